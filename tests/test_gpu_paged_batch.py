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


def test_pool_above_four_gigabytes(L):
    """Pages whose byte offsets pass 32 bits behave as the same pages of a small pool."""
    H, d, P, n = 8, 128, 64, 150
    many = (1 << 32) // (H * P * d) + 40
    ctx = context(L, "bf16", H, 2, d)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(n, H, d, generator=g).bfloat16().cuda() for _ in "kv")
    q = torch.randn(1, 1, 2 * H, d, generator=g).bfloat16().cuda()
    got = []
    for n_pages, first in ((3, 0), (many, many - 3)):
        t = L.alloc_pages(ctx.cfg, n_pages, P, "cuda")
        table = torch.tensor([[first + 2, first, first + 1]], dtype=torch.int32, device="cuda")
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        pages = L.paged_cache(t["k_code"], t["v_code"], t["k_scale"], t["v_scale"], table, lens)
        L.paged_append(ctx, pages, k, v)
        out, lse = torch.empty_like(q), torch.empty(1, 1, 2 * H, device="cuda")
        ws = torch.empty(L.paged_workspace_size(ctx.cfg, 1), dtype=torch.uint8, device="cuda")
        L.paged_attend(ctx, pages, q, out, ws, lse=lse)
        ks, vs = (torch.empty(1, n, H, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        L.paged_gather(ctx, pages, ks, vs)
        assert ctx.last_error() == L.OK
        got.append((out, lse, ks, vs, t["k_scale"][first:first + 3].clone()))
        del t, pages
    assert all(torch.equal(a, b) for a, b in zip(*got))
    ctx.close()


def test_two_streams_at_once(L):
    """One context, two streams, each with its own pages, outputs and workspace: the paged calls
    keep nothing in the context."""
    ctx = context(L, "bf16", 2, 4, 128)
    runs = []
    for i, lens in enumerate(([3000, 17, 900], [5000, 1, 0])):
        c = Case(L, lens, 16, 2, 128, seed=40 + i)
        pages = c.device()
        q = torch.randn(3, 1, 8, 128, generator=torch.Generator().manual_seed(i)).bfloat16().cuda()
        ws = torch.empty(L.paged_workspace_size(ctx.cfg, 3), dtype=torch.uint8, device="cuda")
        alone = torch.empty_like(q)
        L.paged_attend(ctx, pages, q, alone, ws)
        runs.append((c, pages, q, ws, alone, torch.empty_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, pages, q, ws, alone, out, s in runs:
            L.paged_attend(ctx, pages, q, out, ws, stream=s)
    torch.cuda.synchronize()
    assert ctx.last_error() == L.OK
    for c, pages, q, ws, alone, out, s in runs:
        assert torch.equal(alone, out)
    ctx.close()


def test_two_graphs_share_a_workspace(L):
    """An append and an attend captured twice over one workspace, replayed in turns."""
    ctx = context(L, "bf16", 2, 4, 64)
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, 2), dtype=torch.uint8, device="cuda")
    made = []
    for i in range(2):
        c = Case(L, [40 + i, 700 * (i + 1)], 32, 2, 64, seed=50 + i)
        pages = c.device()
        q = torch.randn(2, 1, 8, 64, generator=torch.Generator().manual_seed(i)).bfloat16().cuda()
        k = torch.randn(2, 2, 64, generator=torch.Generator().manual_seed(9 + i)).bfloat16().cuda()
        out, want = torch.empty_like(q), torch.empty_like(q)

        def step(o):
            L.paged_append(ctx, pages, k, k)
            L.paged_attend(ctx, pages, q, o, ws)

        step(want)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(out)
        made.append((g, out, want, c, pages, q, k))
    for _ in range(3):
        for g, *_ in made:
            g.replay()
    torch.cuda.synchronize()
    assert ctx.last_error() == L.OK
    for g, out, want, *_ in made:
        assert torch.equal(out, want)
    ctx.close()


def test_nan_scale_stays_in_its_sequence(L):
    """A sequence with NaN scales (a cache written elsewhere, or never) reaches no other one that the
    same warps take."""
    lens = [16, 20, 16, 40] * 500          # short runs of many sequences in every warp
    c = Case(L, lens, 16, 1, 64, seed=60)
    for b in range(0, len(lens), 4):
        c.ref.scale["v"][c.table[b, 0]] = np.nan
        c.ref.scale["k"][c.table[b, 0]] = np.nan
    pages = c.device()
    ctx = context(L, "bf16", 1, 2, 64)
    q = torch.randn(len(lens), 1, 2, 64, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    out = torch.empty_like(q)
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, len(lens)), dtype=torch.uint8, device="cuda")
    L.paged_attend(ctx, pages, q, out, ws)
    assert ctx.last_error() == L.OK
    nan = torch.isnan(out).flatten(1).any(dim=1).cpu()
    assert nan[0::4].all() and not nan[1::4].any() and not nan[2::4].any() and not nan[3::4].any()
    ctx.close()


def test_oversize_pools_are_refused(L):
    """Sizes whose rows or positions pass the kernels' indices, by descriptor only."""
    import ctypes
    c = Case(L, [20], 16, 8, 128, seed=61)
    pages = c.device()
    ctx = context(L, "bf16", 8, 1, 128)
    q = torch.zeros(1, 1, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(L.paged_workspace_size(ctx.cfg, 1), dtype=torch.uint8, device="cuda")
    for field, value, want in (("n_pages", 1 << 24, L.ERR_UNSUPPORTED), ("max_pages", (1 << 20) + 1, L.ERR_UNSUPPORTED),
                               ("n_seqs", 8193, L.ERR_UNSUPPORTED), ("n_seqs", 0, L.ERR_SHAPE),
                               ("page_tokens", 48, L.ERR_UNSUPPORTED), ("n_pages", 0, L.ERR_SHAPE)):
        p = L.lowram_pages.from_buffer_copy(pages)
        setattr(p, field, value)
        r = ctypes.byref(p)
        assert L.lowram_paged_attend(ctx.handle, r, q.data_ptr(), 1, q.data_ptr(), None, ws.data_ptr(),
                                     ws.numel(), None) == want, field
        assert L.lowram_paged_gather(ctx.handle, r, None, 1, q.data_ptr(), q.data_ptr(), None) == want, field
        assert L.lowram_paged_append(ctx.handle, r, q.data_ptr(), q.data_ptr(), 1024, 1024, 1, None, 1,
                                     None, 1, None) == want, field
    p = L.lowram_pages.from_buffer_copy(pages)
    p.table = p.table + 4
    assert L.lowram_paged_attend(ctx.handle, ctypes.byref(p), q.data_ptr(), 1, q.data_ptr(), None,
                                 ws.data_ptr(), ws.numel(), None) == L.ERR_ALIGN
    p.table = None
    assert L.lowram_paged_attend(ctx.handle, ctypes.byref(p), q.data_ptr(), 1, q.data_ptr(), None,
                                 ws.data_ptr(), ws.numel(), None) == L.ERR_INVALID_ARG
    ctx.close()
