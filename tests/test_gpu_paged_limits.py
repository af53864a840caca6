"""Paged 8-bit cache at the ends of what include/lowram.h admits, against the plain 64-bit
implementation: NaN values that several drafted tokens share, runs of millions of tokens.

The tolerances are those of test_gpu_paged unless a test says otherwise."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged import DT, Case, check_attend, context, f64

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
