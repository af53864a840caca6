"""Paged 8-bit cache at the ends of what include/lowram.h admits, against the plain 64-bit
implementation: NaN values that several drafted tokens share, runs of millions of tokens,
value scales anywhere in 2^-64 .. 2^120, outputs that cancel.

The tolerances are those of test_gpu_paged unless a test says otherwise."""
import numpy as np
import pytest
import torch

from long_context_decode_02_b200 import synth
from tests import paged_reference as R
from tests.test_gpu_decode import prepared
from tests.test_gpu_paged import DT, Case, check_attend, context, f64
from tests.test_gpu_paged_decode import BF16, F32, check_step, new_pages, suffix_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L(cuda_device):
    from long_context_decode_02_b200 import lowram
    return lowram


def attend(L, ctx, pages, q, G):
    """out and lse of q [B][n_q][H_q][d], from a workspace of 0xff bytes."""
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:-1], float("nan"), device="cuda")
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, q.shape[0], q.shape[1]), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    L.paged_attend(ctx, pages, q, out, ws, lse=lse)
    assert ctx.last_error() == L.OK
    return out, lse


@pytest.mark.parametrize("dtype,d,P", [("bf16", 128, 16), ("bf16", 128, 64), ("bf16", 64, 32), ("f32", 64, 16),
                                       ("f32", 128, 32)])
def test_nan_value_in_one_element_of_consecutive_tokens(L, dtype, d, P):
    """The last three tokens hold a NaN in the same elements: every query that sees the first of
    them gets it, whichever token a lane finds last. A second sequence of the same warps has its
    own NaN elements."""
    lens, nq = [36, 71], 4
    c = Case(L, lens, P, 1, d, seed=70)
    for b, els in ((0, (5, d // 2 + 17, d - 1)), (1, (0, 6))):
        for t in range(lens[b] - 3, lens[b]):
            for el in els:
                c.ref.code["v"][c.table[b, t // P], 0, t % P, el] = 0x7f if t & 1 else 0xff
    pages = c.device()
    ctx = context(L, dtype, 1, 2, d)
    q = torch.randn(2, nq, 2, d, generator=torch.Generator().manual_seed(3)).to(DT[dtype]).cuda()
    out, lse = attend(L, ctx, pages, q, 2)
    nan = torch.isnan(out).cpu()
    want = torch.zeros_like(nan)
    for b, els in ((0, (5, d // 2 + 17, d - 1)), (1, (0, 6))):
        want[b, 1:, :, list(els)] = True
    assert torch.equal(nan, want)
    ref = c.ref.attend(c.table, c.lens, f64(q), 2)
    check_attend(dtype, out[:, :1], lse[:, :1], tuple(x[:, :1] for x in ref))
    ctx.close()


def test_long_runs_of_a_warp(L):
    """2^21 tokens of positive values for more (sequence, head)s than the GPU has warps, so a warp
    sums a whole one: its 65536 steps add no bias. The sequences repeat one list of 4096 tokens,
    whose exact result they share; lse is larger by the repetitions' logarithm."""
    P, n, H, seqs = 64, 1 << 21, 8, 148
    c = Case(L, [4096], P, H, 128, seed=71)
    v = c.ref.code["v"] & 0x7f
    c.ref.code["v"] = np.where(v == 0x7f, 0x38, v).astype(np.uint8)
    q = torch.randn(1, 1, H, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    out, lse, absv, zabs = c.ref.attend(c.table, c.lens, f64(q), 1)
    c.table = np.tile(c.table[:, :4096 // P], (seqs, n // 4096))
    c.lens = [n] * seqs
    pages = c.device()
    ctx = context(L, "bf16", H, 1, 128)
    got, got_lse = attend(L, ctx, pages, q.repeat(seqs, 1, 1, 1).cuda(), 1)
    want = (out, lse + np.log(n / 4096), absv, zabs)
    for b in range(0, seqs, 21):
        check_attend("bf16", got[b:b + 1], got_lse[b:b + 1], want, b)
    ctx.close()


def scaled(L, lens, P, H, d, seed, lo, hi, one_element=False):
    """A case whose pages have value scales 2^lo and 2^hi in turn (two of a kind now and then),
    the large ones' codes small enough to stay finite. one_element: a large page has values in
    element 3 only, so that the other elements show what the small pages keep of their digits."""
    c = Case(L, lens, P, H, d, seed=seed)
    g = np.random.default_rng(seed)
    for row, n in zip(c.table, lens):
        for i in range(-(-n // P)):
            big = bool(i & 1) != (g.random() < 0.25)
            c.ref.scale["v"][row[i]] = 2.0 ** (hi if big else lo)
            if big:
                c.ref.code["v"][row[i]] = R.encode(np.clip(R.decode(c.ref.code["v"][row[i]]), -240, 240))
                if one_element:
                    c.ref.code["v"][row[i], ..., :3] = 0
                    c.ref.code["v"][row[i], ..., 4:] = 0
    return c


SCALES = [(-64, 62), (-64, 63), (-64, 84), (-64, 120), (-8, 120), (-20, 14), (-8, 0), (-7, 2)]


@pytest.mark.parametrize("one_element", [False, True])
@pytest.mark.parametrize("dtype,G,d,P,nq,lens", [
    ("bf16", 4, 128, 16, 1, [77, 200]),
    ("bf16", 8, 128, 64, 1, [300]),
    ("bf16", 8, 128, 16, 3, [50, 2]),
    ("bf16", 4, 64, 32, 4, [150]),
    ("bf16", 1, 64, 16, 1, [90]),
    ("f32", 4, 64, 16, 1, [100, 31]),
    ("f32", 4, 128, 32, 2, [150]),
    ("f32", 2, 64, 64, 1, [400]),
])
def test_value_scales_far_apart(L, dtype, G, d, P, nq, lens, one_element):
    """Tokens of about the same weight in pages whose value scales lie anywhere in the admitted
    range: none leaves the softmax's sum, and each element keeps its digits."""
    ctx = context(L, dtype, 2, G, d)
    q = torch.randn(len(lens), nq, 2 * G, d, generator=torch.Generator().manual_seed(d + nq)) / 8
    q = q.to(DT[dtype]).cuda()
    for i, (lo, hi) in enumerate(SCALES):
        c = scaled(L, lens, P, 2, d, 80 + i, lo, hi, one_element)
        out, lse = attend(L, ctx, c.device(), q, G)
        check_attend(dtype, out, lse, c.ref.attend(c.table, c.lens, f64(q), G), (lo, hi))
    ctx.close()


@pytest.mark.parametrize("dtype,d,P", [("bf16", 128, 64), ("bf16", 128, 16), ("f32", 64, 32)])
def test_value_scales_far_apart_over_runs(L, dtype, d, P):
    """The same where a warp's run has several steps and a row many partials."""
    H = 4
    ctx = context(L, dtype, H, 1, d)
    q = torch.randn(2, 1, H, d, generator=torch.Generator().manual_seed(7)).to(DT[dtype]).cuda() / 8
    for lo, hi in ((-64, 63), (-64, 120), (-8, 30)):
        c = scaled(L, [29000, 700], P, H, d, 90, lo, hi, one_element=hi == 30)
        out, lse = attend(L, ctx, c.device(), q, 1)
        check_attend(dtype, out, lse, c.ref.attend(c.table, c.lens, f64(q), 1), (lo, hi))
    ctx.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,H,n", [(16, 1, 64), (64, 1, 2530), (32, 4, 17000)])
def test_tiny_weights_of_huge_values(L, dtype, P, H, n):
    """Logits that give the large pages weights far below what fp16, or one fp32 exponential,
    holds beside 1, though their values make up the output: within a step, over the partials of a
    row, and over a warp's run of steps."""
    d = 64
    for lo, hi, drop in ((-8, 40, 25), (-64, 60, 80), (-64, 119, 112), (-64, 119, 160)):
        for first in (0, 1):
            c = Case(L, [n], P, H, d, seed=99)
            c.ref.code["k"][:] = 0
            c.ref.scale["k"][:] = 1.0
            for i, page in enumerate(c.table[0, :-(-n // P)]):
                big = i % 2 == first
                c.ref.scale["v"][page] = 2.0 ** (hi if big else lo)
                if big:      # z = q k / 8 with q = 4 ln 2: a weight of 2^-drop
                    c.ref.code["k"][page, ..., 0] = R.encode(np.array(-2.0 * drop))
                c.ref.code["v"][page] = R.encode(np.clip(R.decode(c.ref.code["v"][page]), -240, 240))
            # the codes behind the length are NaN still
            if n % P:
                c.ref.code["v"][c.table[0, n // P], :, n % P:, 0] = 0x7f
            q = torch.zeros(1, 1, 2 * H, d)
            q[..., 0] = 4 * np.log(2.0)
            q = q.to(DT[dtype]).cuda()
            ctx = context(L, dtype, H, 2, d)
            out, lse = attend(L, ctx, c.device(), q, 2)
            check_attend(dtype, out, lse, c.ref.attend(c.table, c.lens, f64(q), 2), (lo, hi, drop, first))
            ctx.close()


@pytest.mark.parametrize("sh,exp", [(BF16, 119), (BF16, -60), (F32, 110)])
def test_prefix_beside_far_scales(L, cuda_device, sh, exp):
    """A compressed prefix and a suffix whose values are 2^exp times as large: the softmax spans
    both."""
    dev, P, lens = cuda_device, 16, [3, 40][:sh.batch - 1] + [200]
    t, t_dev, cdev, co, _ = prepared(sh, 0, dev)
    cfg = L.make_config(sh)
    ctx = L.Context(cfg, dev.index or 0)
    params = L.layer_params(*(t_dev[n] for n in ("basis", "w1", "b1", "w2", "b2")))
    pages, pt, table, dlens = new_pages(L, sh, P, max(lens) + 1, dev)
    n = sum(lens)
    g = torch.Generator().manual_seed(97)
    k, v = (torch.randn(n, sh.n_kv_heads, sh.head_dim, generator=g) for _ in "kv")
    v[lens[0]:] *= 2.0 ** exp          # sequence 0 keeps values of the prefix's size
    k, v = k.to(sh.torch_dtype).to(dev), v.to(sh.torch_dtype).to(dev)
    dlens.copy_(torch.tensor(lens, dtype=torch.int32))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
    L.paged_append(ctx, pages, k, v, cu_new=cu, pos_base=torch.full_like(dlens, sh.n_tokens))
    ws = torch.empty(L.decode_paged_workspace_size(cfg), dtype=torch.uint8, device=dev).fill_(255)
    sk, sv = (suffix_values(pt, table, lens, x) for x in "kv")
    check_step(L, sh, ctx, cdev, t, co, params, synth.queries(sh, 0, 0), pages, sk, sv, ws, dev)
    ctx.close()


@pytest.mark.parametrize("G,nq,d", [(4, 1, 128), (1, 1, 64), (2, 2, 64), (1, 4, 128)])
def test_weights_of_up_to_four_bf16_rows(L, G, nq, d):
    """Up to four query rows of a head hold their weights in two fp16 parts, 2^-21 together, as
    fp32 contexts do. It shows where an output cancels: two tokens of weights a and b with values
    near b and -a, so that its own rounding is small beside sum p |v|. Keys and queries have one
    element, which keeps the logits' share of the bound at (d + 8) 2^-22 |z|."""
    seqs, P = 24, 16
    c = Case(L, [nq + 1] * seqs, P, 1, d, seed=72)
    g = np.random.default_rng(73)
    q = torch.zeros(seqs, nq, G, d)
    q[..., 0] = 1.0
    k, v, r = c.ref.code["k"], c.ref.code["v"], c.table[:, 0]
    c.ref.scale["k"][:] = 2.0 ** -3
    k[r, 0, :nq + 1] = 0
    v[r, 0, :nq + 1] = 0
    # the last query's weights: token nq at e^z of the others, token 0 holds the other value
    k[r, 0, nq, 0] = R.encode(-(8.0 + 4.0 * np.arange(seqs)))
    z = R.decode(k[r, 0, nq, 0]) / 8 / d ** 0.5
    first = np.exp2(g.uniform(2, 5.5, size=(seqs, d))) * g.choice([-1, 1], size=(seqs, d))
    v[r, 0, 0] = R.encode(first)
    v[r, 0, nq] = R.encode(-R.decode(v[r, 0, 0]) * np.exp(-z)[:, None])
    pages = c.device()
    ctx = context(L, "bf16", 1, G, d)
    qd = q.bfloat16().cuda()
    out, lse = attend(L, ctx, pages, qd, G)
    want, _, absv, zabs = c.ref.attend(c.table, c.lens, f64(qd), G)
    ez = (d + 8) * 2.0 ** -22 * zabs + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -21 + 2 * ez[..., None]) * absv
    over = np.abs(f64(out) - want) - tol
    assert over.max() <= 0, (over.max(), (over / absv.clip(1e-30)).max())
    ctx.close()
