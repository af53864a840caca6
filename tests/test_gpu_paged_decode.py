"""Decode over the compressed prefix plus a paged 8-bit suffix (lowram_decode_step_paged)
against the oracle's decode_step_with_suffix on the suffix values that the pages hold, and the
whole life of a suffix: appended, attended, read back, compressed and appended to the prefix.

Bars: selections as in the decode tests, outputs within the decode tests' tolerance of their
dtype (the compressed part's error; the pages' own is far below it)."""
import numpy as np
import pytest
import torch

import oracle.lowram_oracle as O
from long_context_decode_02_b200 import synth
from tests import helpers as H
from tests import paged_reference as R
from tests.test_gpu_decode import prepared

pytestmark = pytest.mark.gpu

BF16 = synth.CONFIGS[1].replace(name="paged-bf16", n_tokens=2048, batch=3, seed=91)
F32 = synth.CONFIGS[0].replace(name="paged-f32", n_tokens=512, batch=2, seed=92)
SIMT = synth.CONFIGS[1].replace(name="paged-simt", n_tokens=1024, batch=2, n_kv_heads=2, n_q_heads=4,
                                head_dim=64, rank=32, seed=93)


@pytest.fixture(scope="module")
def L(cuda_device):
    from long_context_decode_02_b200 import lowram
    return lowram


def new_pages(L, sh, P, longest, dev):
    per = -(-longest // P)
    t = L.alloc_pages(L.make_config(sh), sh.batch * per, P, dev)
    table = torch.randperm(sh.batch * per, generator=torch.Generator().manual_seed(5))
    table = table.view(sh.batch, per).to(torch.int32).to(dev)
    lens = torch.zeros(sh.batch, dtype=torch.int32, device=dev)
    return L.paged_cache(t["k_code"], t["v_code"], t["k_scale"], t["v_scale"], table, lens), t, table, lens


def suffix_values(t, table, lens, name):
    ref = R.Pages(*(t[n].cpu().numpy() for n in ("k_code", "v_code", "k_scale", "v_scale")))
    tab = table.cpu().numpy()
    return [ref.values(name, tab[b], int(n)) for b, n in enumerate(lens)]


def check_step(L, sh, ctx, cdev, t, co, params, q, pages, sk, sv, ws, dev):
    k = min(sh.top_k, sh.n_chunks)
    p = H.oracle_params(t)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=dev)
    sel = torch.empty(sh.batch, sh.n_kv_heads, k, dtype=torch.int32, device=dev)
    L.decode_step_paged(ctx, cdev, params, q.to(dev), pages, out, ws, sel_out=sel)
    assert ctx.last_error() == L.OK
    g = sel.cpu().numpy()
    osel, scores = O.select_chunks(H.f64(q), co["landmark"], sh.top_k)
    ties = H.compare_selection(g, osel, scores, k)
    H.assert_ties_bounded(ties, sh.batch * sh.n_kv_heads, "paged decode selection")
    for b in range(sh.batch):
        one = {n: x[b:b + 1] for n, x in co.items()}
        want, _ = O.decode_step_with_suffix(H.f64(q)[b:b + 1], one, p["basis"], p["w1"], p["b1"],
                                            p["w2"], p["b2"], sk[b][None], sv[b][None],
                                            chunk=sh.chunk, top_k=sh.top_k, theta=sh.theta,
                                            act=sh.act, sel=g[b:b + 1].astype(np.int64))
        err = H.rel_err(H.f64(out)[b:b + 1], want)
        assert err <= H.TOL[sh.dtype], (b, err)
    return out


@pytest.mark.parametrize("sh,variant,P,lens", [
    (BF16, "DECODE_TCGEN05", 16, [0, 1, 600]),
    (BF16, "DECODE_SIMT", 64, [70, 0, 64]),
    (BF16, "DECODE_TCGEN05", 32, [0, 0, 0]),
    (F32, "DECODE_AUTO", 16, [33, 200]),
    (SIMT, "DECODE_AUTO", 32, [31, 400]),
])
def test_decode_step_paged_matches_oracle(L, cuda_device, sh, variant, P, lens):
    dev = cuda_device
    t, t_dev, cdev, co, _ = prepared(sh, 0, dev)
    cfg = L.make_config(sh, decode_variant=getattr(L, variant))
    ctx = L.Context(cfg, dev.index or 0)
    params = L.layer_params(*(t_dev[n] for n in ("basis", "w1", "b1", "w2", "b2")))
    pages, pt, table, dlens = new_pages(L, sh, P, max(lens) + 1, dev)
    g = torch.Generator().manual_seed(94)
    n = sum(lens)
    k, v = (torch.randn(n, sh.n_kv_heads, sh.head_dim, generator=g).to(sh.torch_dtype).to(dev) for _ in "kv")
    dlens.copy_(torch.tensor(lens, dtype=torch.int32))
    if n:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
        base = torch.full((sh.batch,), sh.n_tokens, dtype=torch.int32, device=dev)
        L.paged_append(ctx, pages, k, v, cu_new=cu, pos_base=base)
    ws = torch.empty(L.decode_paged_workspace_size(cfg), dtype=torch.uint8, device=dev).fill_(255)
    sk, sv = (suffix_values(pt, table, lens, x) for x in "kv")
    for step in range(2):
        q = synth.queries(sh, 0, step)
        out = check_step(L, sh, ctx, cdev, t, co, params, q, pages, sk, sv, ws, dev)
    if not n:      # no suffix at all: the plain decode step
        ref = torch.empty_like(out)
        L.decode_step(ctx, cdev, params, q.to(dev), ref, ws)
        assert H.rel_err(H.f64(out), H.f64(ref)) <= 2.0 ** -8
    ctx.close()


def test_paged_suffix_agrees_with_dense_suffix(L, cuda_device):
    """The same suffix values in pages and in a dense bf16 buffer: one answer."""
    sh, dev, n = BF16, cuda_device, 500
    t, t_dev, cdev, co, _ = prepared(sh, 0, dev)
    cfg = L.make_config(sh)
    ctx = L.Context(cfg, dev.index or 0)
    params = L.layer_params(*(t_dev[x] for x in ("basis", "w1", "b1", "w2", "b2")))
    pages, pt, table, lens = new_pages(L, sh, 16, n, dev)
    k, v = (torch.randn(sh.batch, n, sh.n_kv_heads, sh.head_dim,
                        generator=torch.Generator().manual_seed(i)).bfloat16().to(dev) for i in (1, 2))
    lens.fill_(n)
    L.paged_append(ctx, pages, k, v, pos_base=torch.full_like(lens, sh.n_tokens))
    ks, vs = torch.empty_like(k), torch.empty_like(v)
    L.paged_gather(ctx, pages, ks, vs)
    q = synth.queries(sh, 0, 3).to(dev)
    a, b = torch.empty_like(q), torch.empty_like(q)
    L.decode_step_paged(ctx, cdev, params, q, pages, a, torch.empty(
        L.decode_paged_workspace_size(cfg), dtype=torch.uint8, device=dev))
    L.decode_step_suffix(ctx, cdev, params, q, ks, vs, n, b, torch.empty(
        L.suffix_workspace_size(cfg, n), dtype=torch.uint8, device=dev))
    assert ctx.last_error() == L.OK
    # Before their last rounding the two differ by the weights' fp16 rounding, 2^-11 sum p |v| over
    # the suffix (at most that of a softmax over the suffix alone); two values that far apart round
    # to bf16 values at most that and one step, 2^-7 of the larger, apart.
    qs = q.double().view(sh.batch, sh.n_kv_heads, sh.group, -1)
    w = torch.softmax(torch.einsum("bhgd,bthd->bhgt", qs, ks.double()) / 128 ** 0.5, dim=-1)
    mean = torch.einsum("bhgt,bthd->bhgd", w, vs.double().abs()).reshape(a.shape)
    tol = 2.0 ** -7 * torch.maximum(a.abs(), b.abs()).double() + 2.0 ** -11 * mean
    over = ((a.double() - b.double()).abs() - tol).max().item()
    assert over <= 0.0
    ctx.close()


def test_life_of_a_suffix(L, cuda_device):
    """Full rank, every token a residual row, every chunk selected, so each step is exact
    attention over what the caches hold: tokens are appended to the pages, decoded over, a block
    of whole chunks read back, compressed at its true positions and appended to the prefix, and
    the rest of the suffix goes on in the pages behind it."""
    dev = cuda_device
    T0, block, rest = 512, 256, 37
    sh = synth.CONFIGS[1].replace(name="paged-life", n_kv_heads=1, n_q_heads=4, rank=128, res_frac=1.0,
                                  top_k=10 ** 6, n_tokens=T0, batch=2, seed=95)
    t = H.stored_layer(sh, 0)
    td = {k: v.to(dev) for k, v in t.items()}
    params = L.layer_params(*(td[n] for n in ("basis", "w1", "b1", "w2", "b2")))
    cfg = L.make_config(sh)
    ctx = L.Context(cfg, dev.index or 0)
    pre = L.alloc_cache(cfg, dev)
    L.encode(ctx, td["k"], td["v"], params, pre,
             torch.empty(L.workspace_size(cfg, L.OP_ENCODE), dtype=torch.uint8, device=dev))
    pages, pt, table, lens = new_pages(L, sh, 16, block + rest, dev)
    g = torch.Generator().manual_seed(96)
    k, v = (torch.randn(sh.batch, block + rest, 1, 128, generator=g).bfloat16().to(dev) for _ in "kv")
    base = torch.full((sh.batch,), T0, dtype=torch.int32, device=dev)
    lens.fill_(block)
    L.paged_append(ctx, pages, k[:, :block].contiguous(), v[:, :block].contiguous(), pos_base=base)
    for i in range(rest):
        lens.add_(1)
        L.paged_append(ctx, pages, k[:, block + i:block + i + 1].contiguous(),
                       v[:, block + i:block + i + 1].contiguous(), pos_base=base)
    q = synth.queries(sh, 0, 0).to(dev)
    before = torch.empty_like(q)
    L.decode_step_paged(ctx, pre, params, q, pages, before, torch.empty(
        L.decode_paged_workspace_size(cfg), dtype=torch.uint8, device=dev))
    assert ctx.last_error() == L.OK
    n = [block + rest] * sh.batch
    dense = O.dense_attention(H.f64(q),
                              np.concatenate([H.f64(t["k"]), np.stack(suffix_values(pt, table, n, "k"))], 1),
                              np.concatenate([H.f64(t["v"]), np.stack(suffix_values(pt, table, n, "v"))], 1))
    assert H.rel_err(H.f64(before), dense) <= 2e-2
    # the block moves from the pages to the compressed prefix
    kb, vb = (torch.empty(sh.batch, block, 1, 128, dtype=torch.bfloat16, device=dev) for _ in "kv")
    L.paged_gather(ctx, pages, kb, vb)
    cfg_b = L.make_config(sh, n_tokens=block, n_res=block, n_positions=T0 + block)
    ctx_b = L.Context(cfg_b, dev.index or 0)
    blk = L.alloc_cache(cfg_b, dev)
    first = T0 // sh.chunk
    blk["chunk_pos"].copy_(torch.arange(first, first + block // sh.chunk, dtype=torch.int32,
                                        device=dev).expand(sh.batch, -1))
    L.encode(ctx_b, kb, vb, params, blk,
             torch.empty(L.workspace_size(cfg_b, L.OP_ENCODE), dtype=torch.uint8, device=dev))
    cfg_d = L.make_config(sh, n_tokens=T0 + block, n_res=T0 + block, n_positions=0)
    ctx_d = L.Context(cfg_d, dev.index or 0)
    dst = L.alloc_cache(cfg_d, dev)
    L.append(ctx_d, dst, ctx, pre, ctx_b, blk)
    # whole pages leave the front of every list; the rest keeps its positions
    tail = table[:, block // 16:].contiguous()
    left = torch.full_like(lens, rest)
    pages2 = L.paged_cache(pt["k_code"], pt["v_code"], pt["k_scale"], pt["v_scale"], tail, left)
    after = torch.empty_like(q)
    L.decode_step_paged(ctx_d, dst, params, q, pages2, after, torch.empty(
        L.decode_paged_workspace_size(cfg_d), dtype=torch.uint8, device=dev))
    assert ctx_d.last_error() == L.OK and ctx_b.last_error() == L.OK
    assert H.rel_err(H.f64(after), dense) <= 2e-2
    for c in (ctx, ctx_b, ctx_d):
        c.close()


def test_decode_step_paged_refusals(L, cuda_device):
    sh, dev = BF16, cuda_device
    cfg = L.make_config(sh)
    ctx = L.Context(cfg, dev.index or 0)
    pages, _, table, lens = new_pages(L, sh, 16, 20, dev)
    cache = {n: x.zero_() for n, x in L.alloc_cache(cfg, dev).items()}
    w = [torch.zeros(s, dtype=torch.bfloat16, device=dev) for s in
         ((1024, 160), (8, 256, 128), (8, 256), (8, 128, 256), (8, 128))]
    params = L.layer_params(*w)
    q = torch.zeros(sh.batch, 32, 128, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(L.decode_paged_workspace_size(cfg), dtype=torch.uint8, device=dev)
    with pytest.raises(L.LowRAMError) as e:
        L.decode_step_paged(ctx, cache, params, q, pages, q.clone(), ws[:1024])
    assert e.value.status == L.ERR_WORKSPACE
    two = L.paged_cache(*pages._refs[:4], table[:2].contiguous(), lens[:2].contiguous())
    with pytest.raises(L.LowRAMError) as e:
        L.decode_step_paged(ctx, cache, params, q, two, q.clone(), ws)
    assert e.value.status == L.ERR_SHAPE
    with pytest.raises(ValueError):
        L.decode_step_paged(ctx, cache, params, q[:2], pages, q[:2].clone(), ws)
    with pytest.raises(ValueError):
        L.decode_step_paged(ctx, cache, params, q.float(), pages, q.float(), ws)
    ctx.close()
