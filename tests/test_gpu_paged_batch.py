"""Paged attend with more sequences than a warp has lanes, and more than a CTA has threads: the
list of steps crosses many short sequences in a warp's run."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged import DT, Case, check_attend, context, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L(cuda_device):
    from long_context_decode_02_b200 import lowram
    return lowram


@pytest.mark.parametrize("dtype,n,H,G,d,P,nq,top", [
    ("bf16", 33, 2, 4, 128, 16, 1, 90),
    ("bf16", 300, 1, 4, 64, 16, 2, 70),
    ("f32", 70, 1, 2, 64, 32, 1, 200),
    ("bf16", 64, 4, 8, 128, 64, 3, 150),
])
def test_many_sequences(L, dtype, n, H, G, d, P, nq, top):
    g = np.random.default_rng(n)
    lens = [int(x) for x in g.integers(0, top, size=n)]
    lens[0] = lens[n // 2] = 0
    c = Case(L, lens, P, H, d, seed=n)
    pages = c.device()
    ctx = context(L, dtype, H, G, d)
    q = torch.randn(n, nq, H * G, d, generator=torch.Generator().manual_seed(n)).to(DT[dtype]).cuda()
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:-1], float("nan"), device="cuda")
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, n, nq), dtype=torch.uint8, device="cuda").fill_(255)
    L.paged_attend(ctx, pages, q, out, ws, lse=lse)
    assert ctx.last_error() == L.OK
    check_attend(dtype, out, lse, c.ref.attend(c.table, c.lens, f64(q), G))
    ctx.close()


def test_all_empty(L):
    """Every sequence empty: zeros, -inf, and nothing else is read."""
    for n in (1, 40):
        c = Case(L, [0] * n, 16, 2, 64, seed=1)
        pages = c.device()
        ctx = context(L, "bf16", 2, 2, 64)
        q = torch.randn(n, 2, 4, 64).bfloat16().cuda()
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:-1], 1.0, device="cuda")
        ws = torch.empty(L.paged_workspace_size(ctx.cfg, n, 2), dtype=torch.uint8, device="cuda")
        L.paged_attend(ctx, pages, q, out, ws, lse=lse)
        assert ctx.last_error() == L.OK
        assert (out == 0).all() and torch.isneginf(lse).all()
        ctx.close()
