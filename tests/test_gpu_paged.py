"""Paged 8-bit cache on the GPU (append, attend, gather) through the public binding, against
the plain 64-bit implementation.

Tolerances, fixed before the first run. u(t) = eps(t)/2 is a rounding's largest relative error.
  append: the scales are equal; a code is the one of the exact value, or of that value moved by
    the largest error of the rotation: 2^-50 of the pair for its fp64 arithmetic, position *
    2^-52 for its angle's rounding, 2^-24 for the rounding to fp32 before the code's.
  attend: weights are rounded to fp16 (bf16 contexts: 2^-11; fp32: two parts, 2^-21 with the
    sums); logits are fp32 sums of d products, each step off by at most 2^-23 of the partial
    sums, (d + 8) 2^-22 sum |q_i k_i| / sqrt(d) in all, and move a weight by that much; the
    exponential adds 2^-20. So
      |out - exact| <= u |exact| + (w + 2 e_z) sum p |v|,   e_z = (d + 8) 2^-22 zabs + 2^-20,
      |lse - exact| <= e_z + 2^-22 |exact| + w.
  gather: equal (a scaled code is exact in both types).
"""
import numpy as np
import pytest
import torch

from tests import paged_reference as R

pytestmark = pytest.mark.gpu

THETA = 5e5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def L(cuda_device):
    from long_context_decode_02_b200 import lowram
    return lowram


def context(L, dtype, H, G, d, batch=1):
    cfg = L.lowram_config(batch=batch, n_tokens=16, n_kv_heads=H, n_q_heads=H * G, head_dim=d,
                          rank=16, chunk=1, mlp_hidden=128, top_k=1, n_res=0, act=L.ACT_SILU,
                          dtype=L.DTYPE_BF16 if dtype == "bf16" else L.DTYPE_F32,
                          decode_variant=L.DECODE_AUTO, res_format=L.RES_STORE, n_positions=0,
                          reserved=0, rope_theta=THETA)
    return L.Context(cfg, 0)


class Case:
    """A cache with random contents, garbage (NaN codes among it) behind every length, and a
    shuffled page list whose unused entries are out of range."""

    def __init__(self, L, lens, P, H, d, seed, spread=3, zero_page=False, shared=False):
        g = np.random.default_rng(seed)
        self.lens = list(lens)
        used = [-(-n // P) for n in lens]
        self.n_pages = sum(used) + 2
        shape = (self.n_pages, H, P, d)
        code = {n: R.encode(np.clip(g.normal(size=shape) * 80, -448, 448)) for n in "kv"}
        scale = {n: 2.0 ** g.integers(-8 - spread, -8 + spread, size=shape[:2]) for n in "kv"}
        order = g.permutation(self.n_pages)
        self.table = np.full((len(lens), max(used + [1]) + 1), -7, np.int32)
        at = 0
        for b, k in enumerate(used):
            self.table[b, :k] = order[at:at + k]
            at += k
            if lens[b] % P:
                for n in "kv":
                    tail = code[n][self.table[b, k - 1], :, lens[b] % P:]
                    tail[...] = g.integers(0, 256, size=tail.shape)
                    tail[..., 0] = 0x7f
        if shared and len(lens) > 1 and used[0] and used[1]:
            self.table[1, 0] = self.table[0, 0]          # a common first page
        if zero_page and used[0]:
            code["v"][self.table[0, 0]] = 0
            scale["v"][self.table[0, 0]] = 2.0 ** -64
        self.ref = R.Pages(code["k"], code["v"], scale["k"], scale["v"])
        self.L = L

    def device(self):
        t = lambda x, dt: torch.from_numpy(np.ascontiguousarray(x)).to(dt).cuda()  # noqa: E731
        r = self.ref
        self.t = [t(r.code["k"], torch.uint8), t(r.code["v"], torch.uint8),
                  t(r.scale["k"], torch.float32), t(r.scale["v"], torch.float32),
                  t(self.table, torch.int32), t(np.array(self.lens), torch.int32)]
        return self.L.paged_cache(*self.t)


def f64(t):
    return t.detach().double().cpu().numpy()


def check_attend(dtype, got, lse, ref, what=""):
    out, want_lse, absv, zabs = ref
    d = out.shape[-1]
    u = torch.finfo(DT[dtype]).eps / 2
    w = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    ez = (d + 8) * 2.0 ** -22 * zabs + 2.0 ** -20
    tol = u * np.abs(out) + (w + 2 * ez[..., None]) * absv
    err = np.abs(f64(got) - out)
    assert np.all(err <= tol), (what, float((err - tol).max()), float(err.max()))
    if lse is not None:
        gl = f64(lse)
        none = np.isinf(want_lse)
        assert np.array_equal(np.isneginf(gl), none), what
        e = np.abs(np.where(none, 0, gl) - np.where(none, 0, want_lse))
        assert np.all(e <= ez + 2.0 ** -22 * np.abs(np.where(none, 0, want_lse)) + w), what


ATTEND = [
    # dtype, H, G, d, P, n_q, lens
    ("bf16", 2, 4, 128, 16, 1, [1]),
    ("bf16", 1, 1, 128, 16, 1, [15, 16, 17, 0, 33]),
    ("bf16", 8, 4, 128, 16, 1, [700, 1, 0, 255, 257]),
    ("bf16", 2, 8, 128, 64, 1, [63, 64, 65, 129]),
    ("bf16", 2, 2, 128, 32, 3, [2, 3, 31, 64, 500]),        # two queries see nothing in the first
    ("bf16", 2, 4, 128, 16, 5, [4, 5, 6, 1000]),
    ("bf16", 1, 8, 128, 32, 16, [7, 16, 300]),
    ("bf16", 3, 4, 64, 16, 1, [1, 31, 32, 333]),
    ("bf16", 2, 8, 64, 64, 2, [100, 0, 1500]),
    ("bf16", 1, 1, 64, 32, 16, [40, 15]),
    ("f32", 2, 4, 64, 16, 1, [1, 77, 0, 300]),
    ("f32", 1, 8, 64, 64, 1, [1000, 63]),
    ("f32", 2, 1, 128, 16, 1, [17, 400]),
    ("f32", 2, 4, 128, 32, 4, [3, 4, 90]),
    ("f32", 1, 2, 64, 16, 16, [20, 129]),
    ("bf16", 4, 4, 128, 16, 1, list(range(0, 66, 5))),
    ("bf16", 2, 8, 64, 32, 5, [4, 77, 600]),                # 40 rows a head: groups of 24
    ("bf16", 2, 2, 128, 64, 11, [10, 300]),
    ("bf16", 1, 4, 128, 16, 6, [0, 5, 47, 48, 49]),
    ("bf16", 2, 4, 64, 16, 4, [33, 2, 260]),                # 16 rows
]


@pytest.mark.parametrize("dtype,H,G,d,P,nq,lens", ATTEND)
def test_attend(L, dtype, H, G, d, P, nq, lens):
    c = Case(L, lens, P, H, d, seed=len(lens) * 100 + nq)
    pages = c.device()
    ctx = context(L, dtype, H, G, d)
    g = torch.Generator().manual_seed(nq + d)
    q = torch.randn(len(lens), nq, H * G, d, generator=g).to(DT[dtype]).cuda()
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:-1], float("nan"), device="cuda")
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, len(lens), nq), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    L.paged_attend(ctx, pages, q, out, ws, lse=lse)
    assert ctx.last_error() == L.OK
    check_attend(dtype, out, lse, c.ref.attend(c.table, c.lens, f64(q), G))
    # without lse, and twice: the same bits
    again = torch.full_like(q, float("nan"))
    L.paged_attend(ctx, pages, q, again, ws)
    assert torch.equal(out, again)
    ctx.close()


def test_attend_long_sequence_and_shared_pages(L):
    lens = [20011, 20010, 5]
    c = Case(L, lens, 32, 2, 128, seed=5, shared=True)
    pages = c.device()
    ctx = context(L, "bf16", 2, 4, 128)
    q = torch.randn(3, 1, 8, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = torch.empty_like(q)
    lse = torch.empty(3, 1, 8, device="cuda")
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, 3), dtype=torch.uint8, device="cuda")
    L.paged_attend(ctx, pages, q, out, ws, lse=lse)
    assert ctx.last_error() == L.OK
    check_attend("bf16", out, lse, c.ref.attend(c.table, c.lens, f64(q), 4))
    ctx.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qscale", [0.0, 2.0 ** -100, 30.0])
def test_attend_magnitudes(L, dtype, qscale):
    """Queries of zero, tiny, and large enough that one token takes the whole weight; value
    scales far apart; a page of zeros."""
    c = Case(L, [250, 90], 16, 2, 64, seed=9, spread=7, zero_page=True)
    pages = c.device()
    ctx = context(L, dtype, 2, 4, 64)
    q = (torch.randn(2, 1, 8, 64, generator=torch.Generator().manual_seed(2)) * qscale).to(DT[dtype]).cuda()
    out = torch.empty_like(q)
    lse = torch.empty(2, 1, 8, device="cuda")
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, 2), dtype=torch.uint8, device="cuda")
    L.paged_attend(ctx, pages, q, out, ws, lse=lse)
    assert ctx.last_error() == L.OK
    check_attend(dtype, out, lse, c.ref.attend(c.table, c.lens, f64(q), 4))
    ctx.close()


def test_attend_value_scales_apart(L):
    """A page whose values are 2^90 larger but whose keys give it no weight must not cost the
    other page its digits; and the other way round."""
    for big in (0, 1):
        c = Case(L, [32], 16, 1, 64, seed=12)
        pg = c.table[0]
        q = torch.ones(1, 1, 1, 64)
        c.ref.code["k"][pg[big]] = R.encode(np.full((1, 16, 64), -448.0))
        c.ref.code["k"][pg[1 - big]] = R.encode(np.full((1, 16, 64), 448.0))
        c.ref.scale["k"][:] = 2.0 ** -3                       # logits +-448: weight e^-896
        c.ref.scale["v"][pg[big]] = 2.0 ** 84
        c.ref.scale["v"][pg[1 - big]] = 2.0 ** -6
        pages = c.device()
        for dtype in ("bf16", "f32"):
            ctx = context(L, dtype, 1, 1, 64)
            qd = q.to(DT[dtype]).cuda()
            out = torch.empty_like(qd)
            ws = torch.empty(L.paged_workspace_size(ctx.cfg, 1), dtype=torch.uint8, device="cuda")
            L.paged_attend(ctx, pages, qd, out, ws)
            assert ctx.last_error() == L.OK
            check_attend(dtype, out, None, c.ref.attend(c.table, c.lens, f64(qd), 1))
            ctx.close()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("slope", [0.02, 0.11, 0.5, -0.11])
def test_attend_rising_logits(L, dtype, d, slope):
    """Logits that rise (or fall) steadily along the sequence, by a little or by far more than a
    reference's slack every few tokens."""
    n = 700
    c = Case(L, [n], 16, 1, d, seed=15, spread=1)
    order = c.table[0, :-(-n // 16)]
    t = np.arange(len(order) * 16, dtype=np.float64).reshape(-1, 16)
    k = np.zeros((c.n_pages, 1, 16, d))
    k[order, 0, :, 0] = np.floor(t * slope * 16) / 16 % 256     # what the 8-bit value leaves is in element 1
    k[order, 0, :, 1] = np.floor(t * slope * 16) / 16 // 256 * 256
    c.ref.code["k"] = R.encode(np.clip(k, -448, 448))
    c.ref.scale["k"][:] = 1.0
    pages = c.device()
    ctx = context(L, dtype, 1, 2, d)
    q = torch.zeros(1, 1, 2, d)
    q[..., 0] = q[..., 1] = d ** 0.5
    q[:, :, 1, 2:] = torch.randn(d - 2, generator=torch.Generator().manual_seed(1)) * 0.1
    q = q.to(DT[dtype]).cuda()
    out, lse = torch.empty_like(q), torch.empty(1, 1, 2, device="cuda")
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, 1), dtype=torch.uint8, device="cuda")
    L.paged_attend(ctx, pages, q, out, ws, lse=lse)
    assert ctx.last_error() == L.OK
    check_attend(dtype, out, lse, c.ref.attend(c.table, c.lens, f64(q), 2))
    ctx.close()


def test_attend_nan_only_reaches_its_rows(L):
    """A NaN key of a valid token reaches the rows that see it and no others."""
    c = Case(L, [40, 40], 16, 1, 128, seed=13)
    c.ref.code["k"][c.table[0, 2], 0, 7, 5] = 0x7f            # token 39 of sequence 0
    pages = c.device()
    ctx = context(L, "bf16", 1, 2, 128)
    q = torch.randn(2, 2, 2, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    out = torch.empty_like(q)
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, 2, 2), dtype=torch.uint8, device="cuda")
    L.paged_attend(ctx, pages, q, out, ws)
    assert torch.isnan(out[0, 1]).all() and torch.isfinite(out[0, 0]).all()
    assert torch.isfinite(out[1]).all()
    ctx.close()


def test_attend_nan_value_of_a_drafted_token(L):
    """A NaN value of a token that only the later queries see stays out of the earlier ones."""
    for dtype, d, P in (("bf16", 128, 16), ("bf16", 64, 32), ("f32", 64, 16), ("f32", 128, 64)):
        c = Case(L, [36, 50], P, 1, d, seed=14)
        c.ref.code["v"][c.table[0, 34 // P], 0, 34 % P, 5] = 0xff
        c.ref.code["v"][c.table[0, 35 // P], 0, 35 % P, 8] = 0x7f
        pages = c.device()
        ctx = context(L, dtype, 1, 2, d)
        q = torch.randn(2, 4, 2, d, generator=torch.Generator().manual_seed(3)).to(DT[dtype]).cuda()
        out = torch.empty_like(q)
        ws = torch.empty(L.paged_workspace_size(ctx.cfg, 2, 4), dtype=torch.uint8, device="cuda")
        L.paged_attend(ctx, pages, q, out, ws)
        assert ctx.last_error() == L.OK
        nan = torch.isnan(out).cpu()
        want = torch.zeros_like(nan)
        want[0, 2:, :, 5] = True
        want[0, 3:, :, 8] = True
        assert torch.equal(nan, want), (dtype, d)
        ref = c.ref.attend(c.table, c.lens, f64(q), 2)
        check_attend(dtype, out[:, :2], None, tuple(x[:, :2] for x in ref))
        ctx.close()


def check_append(c, wrote, t, base, d):
    """Codes and scales on the device against the reference, and untouched bytes."""
    for name, code, scale in (("k", t[0], t[2]), ("v", t[1], t[3])):
        assert np.array_equal(f64(scale), c.ref.scale[name]), name
        got, want = code.cpu().numpy(), c.ref.code[name]
        off = (got != want) & ~((got & 127 == 127) & (want & 127 == 127))
        if off.any():
            x, s = wrote[name], c.ref.scale[name][:, :, None, None] * np.ones_like(wrote[name])
            assert np.isfinite(x[off]).all(), f"{name}: {off.sum()} codes differ outside the new rows"
            pair = np.sqrt(x ** 2 + np.roll(x, d // 2, axis=-1) ** 2)
            e = (2.0 ** -50 + base * 2.0 ** -52) * pair + 2.0 ** -24 * np.abs(x)
            ok = (got == R.encode(np.clip((x - e) / s, -448, 448))) | (got == R.encode(np.clip((x + e) / s, -448, 448)))
            assert ok[off].all(), f"{name}: {(~ok[off]).sum()} codes beyond the rotation's error"


APPEND = [
    # dtype, H, d, P, lens, counts (None: uniform over cu_new = NULL), base
    ("f32", 2, 64, 16, [301], [1], 0),
    ("bf16", 8, 128, 16, [1, 16, 17, 4100], [1, 1, 1, 1], 32768),
    ("bf16", 3, 128, 64, [64, 65, 130, 9], [64, 1, 100, 0], 5),
    ("bf16", 2, 64, 32, [31, 40, 500], [31, 9, 470], (1 << 24) - 600),
    ("f32", 5, 128, 32, [33, 100], [33, 70], 131072),
    ("f32", 1, 64, 64, [200, 7, 64], [137, 7, 1], 0),
    ("bf16", 4, 128, 16, [50, 50], [50, 50], 0),
]


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("dtype,H,d,P,lens,counts,base", APPEND)
def test_append(L, dtype, H, d, P, lens, counts, base, rotate):
    c = Case(L, lens, P, H, d, seed=sum(lens))
    c.ref.scale["k"] *= 2.0 ** -3          # so that earlier codes are rounded again in some pages
    pages = c.device()
    ctx = context(L, dtype, H, 1, d)
    g = torch.Generator().manual_seed(sum(counts))
    n = sum(counts)
    k, v = (torch.randn(n, H, d, generator=g) * torch.exp(torch.randn(n, 1, 1, generator=g)) for _ in "kv")
    k, v = k.to(DT[dtype]), v.to(DT[dtype])
    bases = [base + 11 * b for b in range(len(lens))]
    wrote = c.ref.append(c.table, c.lens, f64(k), f64(v), counts, bases, THETA, rotate)
    uniform = len(set(counts)) == 1
    cu = None if uniform else torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    pb = torch.tensor(bases, dtype=torch.int32, device="cuda")
    for _ in range(2):      # the second call changes nothing
        L.paged_append(ctx, pages, k.cuda(), v.cuda(), cu_new=cu, max_new=max(counts), pos_base=pb,
                       rotate=rotate)
        assert ctx.last_error() == L.OK
        check_append(c, wrote, c.t, max(bases) + max(lens), d)
    ctx.close()


def test_append_special_values(L):
    """Zeros, infinities, NaN, subnormals and the largest values."""
    H, d, P = 2, 64, 16
    for dtype in ("bf16", "f32"):
        c = Case(L, [40], P, H, d, seed=21)
        pages = c.device()
        ctx = context(L, dtype, H, 1, d)
        k = torch.randn(40, H, d, generator=torch.Generator().manual_seed(4))
        k[0:16] = 0
        k[16:32, 0] = 1e-39
        k[16, 1, 3], k[17, 1, 4], k[18, 1, 5] = float("inf"), float("-inf"), float("nan")
        k[32:, 0] = 3.3e38
        k = k.to(DT[dtype])
        c.ref.append(c.table, c.lens, f64(k), f64(k), [40], [0], THETA, False)
        L.paged_append(ctx, pages, k.cuda(), k.cuda(), rotate=False)
        assert ctx.last_error() == L.OK
        for name, code, scale in (("k", c.t[0], c.t[2]), ("v", c.t[1], c.t[3])):
            assert np.array_equal(f64(scale), c.ref.scale[name])
            assert np.array_equal(R.decode(code.cpu().numpy()), R.decode(c.ref.code[name]), equal_nan=True)
        # a rotated infinity is not finite: both elements of its pair are NaN codes, no scale moves
        L.paged_append(ctx, pages, k.cuda(), k.cuda(), rotate=True)
        assert ctx.last_error() == L.OK
        row = c.t[0][c.table[0, 1], 1, 0].cpu().numpy()
        assert row[3] & 127 == 127 and row[3 + d // 2] & 127 == 127
        ctx.close()


def test_append_strided_rows(L):
    """Keys and values as slices of one fused projection output."""
    H, d, P = 2, 128, 16
    c = Case(L, [70, 30], P, H, d, seed=22)
    pages = c.device()
    ctx = context(L, "bf16", H, 4, d)
    fused = torch.randn(100, 8 + 2 * H, d, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    k, v = fused[:, 8:8 + H], fused[:, 8 + H:]
    wrote = c.ref.append(c.table, c.lens, f64(k), f64(v), [70, 30], [0, 0], THETA)
    cu = torch.tensor([0, 70, 100], dtype=torch.int32, device="cuda")
    L.paged_append(ctx, pages, k, v, cu_new=cu)
    assert ctx.last_error() == L.OK
    check_append(c, wrote, c.t, 100, d)
    with pytest.raises(ValueError):     # heads of a token not dense
        L.paged_append(ctx, pages, fused[:, ::2][:, :H], v, cu_new=cu)
    ctx.close()


def test_append_nothing(L):
    c = Case(L, [5, 0], 16, 1, 64, seed=23)
    pages = c.device()
    ctx = context(L, "f32", 1, 1, 64)
    before = [x.clone() for x in c.t]
    none = torch.empty(0, 1, 64, device="cuda")
    L.paged_append(ctx, pages, none, none)
    L.paged_append(ctx, pages, none, none, cu_new=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert ctx.last_error() == L.OK
    assert all(torch.equal(a, b) for a, b in zip(before, c.t))
    ctx.close()


@pytest.mark.parametrize("what", ["cu", "cu_range", "max_new", "len_short", "len_long", "position", "page"])
def test_append_malformed_sequence_is_left_alone(L, what):
    """One of three sequences is malformed: it is reported and left alone, the others are
    written."""
    H, d, P, lens = 2, 64, 16, [20, 20, 20]
    c = Case(L, lens, P, H, d, seed=24)
    k = torch.randn(60, H, d, generator=torch.Generator().manual_seed(6))
    cu, base, max_new = [0, 20, 40, 60], [0, 0, 0], 20
    if what == "cu":
        cu = [0, 20, 15, 60]                     # sequence 1: negative count; 2: 45 tokens
    elif what == "cu_range":
        cu = [0, 20, 40, 61]
    elif what == "max_new":
        cu, max_new = [0, 20, 36, 60], 20        # sequence 2 has 24
    elif what == "position":
        base = [0, 0, (1 << 24) - 10]
    pages = c.device()
    before = [x.clone() for x in c.t[:4]]
    if what == "len_short":
        c.t[5][2] = 19
    elif what == "len_long":
        c.t[5][2] = c.table.shape[1] * P + 1
    elif what == "page":
        c.t[4][2, 0] = c.n_pages
    ctx = context(L, "f32", H, 1, d)
    L.paged_append(ctx, pages, k.cuda(), k.cuda(), cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                   max_new=max_new, pos_base=torch.tensor(base, dtype=torch.int32, device="cuda"))
    assert ctx.last_error() == L.ERR_DEVICE_CHECK
    assert ctx.last_error() == L.OK
    for x, y in zip(before[:2], c.t[:2]):
        assert torch.equal(x[c.table[2, 0]], y[c.table[2, 0]])            # malformed: as it was
        assert not torch.equal(x[c.table[0, 0]], y[c.table[0, 0]])        # the first one: written
    ctx.close()


def test_attend_and_gather_report_bad_pages_and_lengths(L):
    H, d, P, lens = 1, 128, 16, [40, 40]
    c = Case(L, lens, P, H, d, seed=25)
    pages = c.device()
    ctx = context(L, "bf16", H, 1, d)
    c.t[4][0, 1] = -1                            # tokens 16..31 of sequence 0
    q = torch.randn(2, 1, 1, d, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    out, ws = torch.empty_like(q), torch.empty(L.paged_workspace_size(ctx.cfg, 2), dtype=torch.uint8, device="cuda")
    L.paged_attend(ctx, pages, q, out, ws)
    assert ctx.last_error() == L.ERR_DEVICE_CHECK
    # the page's tokens are masked
    keep = [c.table[0, 0], c.table[0, 2]]
    ref = c.ref.attend([keep, c.table[1]], [24, 40], f64(q), 1)
    check_attend("bf16", out, None, ref)
    k, v = (torch.full((2, 40, H, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    L.paged_gather(ctx, pages, k, v)
    assert ctx.last_error() == L.ERR_DEVICE_CHECK
    assert (k[0, 16:32] == 0).all() and np.array_equal(f64(k[1]), c.ref.values("k", c.table[1], 40))
    # lengths out of range are cut
    c.t[4][0, 1] = int(c.table[0, 1])
    c.t[5][0] = -3
    L.paged_attend(ctx, pages, q, out, ws)
    assert ctx.last_error() == L.ERR_DEVICE_CHECK
    assert (out[0] == 0).all()
    ctx.close()


@pytest.mark.parametrize("dtype,H,d,P,lens,start,n", [
    ("bf16", 8, 128, 16, [100, 40, 0, 7], [0, 0, 0, 0], 64),
    ("bf16", 2, 64, 32, [500, 33], [31, -5], 100),
    ("f32", 3, 128, 64, [130, 64], [63, 100], 65),
    ("f32", 1, 64, 16, [17], [16], 1),
])
def test_gather(L, dtype, H, d, P, lens, start, n):
    c = Case(L, lens, P, H, d, seed=n)
    pages = c.device()
    ctx = context(L, dtype, H, 1, d)
    k, v = (torch.full((len(lens), n, H, d), float("nan"), dtype=DT[dtype], device="cuda") for _ in "kv")
    L.paged_gather(ctx, pages, k, v, start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    assert ctx.last_error() == L.OK
    for name, got in (("k", k), ("v", v)):
        for b in range(len(lens)):
            want = np.zeros((n, H, d))
            whole = c.ref.values(name, c.table[b], lens[b])
            for i in range(n):
                if 0 <= start[b] + i < lens[b]:
                    want[i] = whole[start[b] + i]
            assert np.array_equal(f64(got[b]), want), (name, b)
    ctx.close()


def _fresh(L, seqs, P, H, d, longest):
    """An empty cache of NaN codes with pages for `longest` tokens of every sequence."""
    per = -(-longest // P)
    t = [torch.full((seqs * per, H, P, d), 0x7f, dtype=torch.uint8, device="cuda") for _ in "kv"]
    s = [torch.full((seqs * per, H), float("nan"), device="cuda") for _ in "kv"]
    order = torch.randperm(seqs * per, generator=torch.Generator().manual_seed(8))
    table = order.view(seqs, per).to(torch.int32).cuda()
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    return L.paged_cache(t[0], t[1], s[0], s[1], table, lens), t, s, table, lens


@pytest.mark.parametrize("dtype,H,G,d,P", [("bf16", 2, 4, 128, 16), ("f32", 2, 2, 64, 32)])
def test_generation_loop(L, dtype, H, G, d, P):
    """As a user runs them: ragged prompts appended, then one token a step appended and
    attended, the step captured once into a CUDA graph on its own stream and replayed with the
    lengths advanced on the device; the last block gathered for compression."""
    seqs, steps, prompts = 3, 20, [37, 1, 60]
    pages, t, s, table, lens = _fresh(L, seqs, P, H, d, 128)
    ctx = context(L, dtype, H, G, d, batch=seqs)
    g = torch.Generator().manual_seed(9)
    total = sum(prompts) + seqs * steps
    k_all, v_all = (torch.randn(total, H, d, generator=g).to(DT[dtype]) for _ in "kv")
    q_all = torch.randn(steps, seqs, H * G, d, generator=g).to(DT[dtype])
    base = torch.tensor([1000, 2000, 3000], dtype=torch.int32, device="cuda")
    ref = R.Pages(t[0].cpu().numpy(), t[1].cpu().numpy(), s[0].cpu().numpy(), s[1].cpu().numpy())
    tab = table.cpu().numpy()
    n0 = sum(prompts)
    lens.copy_(torch.tensor(prompts, dtype=torch.int32))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), dtype=torch.int32, device="cuda")
    L.paged_append(ctx, pages, k_all[:n0].cuda(), v_all[:n0].cuda(), cu_new=cu, max_new=60, pos_base=base)
    ref.append(tab, prompts, f64(k_all[:n0]), f64(v_all[:n0]), prompts, [1000, 2000, 3000], THETA)
    k_in, v_in = (torch.empty(seqs, 1, H, d, dtype=DT[dtype], device="cuda") for _ in "kv")
    q_in = torch.empty(seqs, H * G, d, dtype=DT[dtype], device="cuda")
    out = torch.empty_like(q_in)
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, seqs), dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(1)
        L.paged_append(ctx, pages, k_in, v_in, pos_base=base)
        L.paged_attend(ctx, pages, q_in, out, ws)

    side = torch.cuda.Stream()
    graph = None
    for i in range(steps):
        rows = slice(n0 + i * seqs, n0 + (i + 1) * seqs)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            k_in.copy_(k_all[rows, None])
            v_in.copy_(v_all[rows, None])
            q_in.copy_(q_all[i])
            if i == 3:
                side.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step()
            if graph is None:
                step()
            else:
                graph.replay()
        side.synchronize()
        now = [p + i + 1 for p in prompts]
        ref.append(tab, now, f64(k_all[rows]), f64(v_all[rows]), [1] * seqs, [1000, 2000, 3000], THETA)
        if i in (0, 2, 3, 4, 12, steps - 1):
            assert ctx.last_error() == L.OK
            check_attend(dtype, out, None,
                         tuple(x[:, 0] for x in ref.attend(tab, now, f64(q_all[i])[:, None], G)), f"step {i}")
    for x, name in ((0, "k"), (1, "v")):
        assert np.array_equal(f64(s[x])[np.isfinite(f64(s[x]))], ref.scale[name][np.isfinite(ref.scale[name])])
    k_out, v_out = (torch.empty(seqs, 16, H, d, dtype=DT[dtype], device="cuda") for _ in "kv")
    L.paged_gather(ctx, pages, k_out, v_out)
    assert ctx.last_error() == L.OK
    for b in range(seqs):
        assert np.array_equal(f64(k_out[b]), ref.values("k", tab[b], 16))
        assert np.array_equal(f64(v_out[b]), ref.values("v", tab[b], 16))
    ctx.close()


def test_refusals(L):
    H, G, d, P = 2, 4, 64, 16
    c = Case(L, [20, 20], P, H, d, seed=30)
    pages = c.device()
    ctx = context(L, "bf16", H, G, d)
    q = torch.zeros(2, 1, H * G, d, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, 1, H * G, device="cuda")
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, 2), dtype=torch.uint8, device="cuda")
    k = torch.zeros(2, H, d, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: L.paged_attend(ctx, pages, q.float(), out, ws),
                lambda: L.paged_attend(ctx, pages, q[:1], out[:1], ws),
                lambda: L.paged_attend(ctx, pages, q, out, ws, lse=lse.double()),
                lambda: L.paged_attend(ctx, pages, q.cpu(), out, ws),
                lambda: L.paged_attend(ctx, pages, q[..., ::2].repeat(1, 1, 1, 2).transpose(2, 3), out, ws),
                lambda: L.paged_append(ctx, pages, k.float(), k),
                lambda: L.paged_append(ctx, pages, k[:, :1], k[:, :1]),
                lambda: L.paged_append(ctx, pages, k, k, cu_new=torch.zeros(2, dtype=torch.int32, device="cuda")),
                lambda: L.paged_append(ctx, pages, k, k, pos_base=torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: L.paged_gather(ctx, pages, k, k)):
        with pytest.raises(ValueError):
            bad()
    status = lambda f: pytest.raises(L.LowRAMError, f).value.status  # noqa: E731
    assert status(lambda: L.paged_attend(ctx, pages, q, out, ws[:64])) == L.ERR_WORKSPACE
    assert status(lambda: L.paged_append(ctx, pages, torch.cat([k, k])[:3], torch.cat([k, k])[:3])) == L.ERR_SHAPE
    big = torch.zeros(2, 17, H * G, d, dtype=torch.bfloat16, device="cuda")
    assert status(lambda: L.paged_attend(ctx, pages, big, big.clone(), ws)) == L.ERR_UNSUPPORTED
    odd = torch.zeros(2, H * d + 4, dtype=torch.bfloat16, device="cuda")[:, :H * d].unflatten(1, (H, d))
    assert status(lambda: L.paged_append(ctx, pages, odd, odd)) == L.ERR_ALIGN
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    assert status(lambda: L.paged_append(ctx, pages, k, k, cu_new=cu, max_new=3)) == L.ERR_SHAPE
    t = list(c.t)
    t[0], t[1] = (torch.zeros(4, H, 8, d, dtype=torch.uint8, device="cuda") for _ in "kv")
    t[2], t[3] = (torch.zeros(4, H, device="cuda") for _ in "kv")
    assert status(lambda: L.paged_attend(ctx, L.paged_cache(*t), q, out, ws)) == L.ERR_UNSUPPORTED
    assert ctx.last_error() == L.OK
    ctx.close()
