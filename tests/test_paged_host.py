"""Paged 8-bit cache, host side: the reference's own pins and every refusal that needs no
GPU (workspace sizes, descriptor checks)."""
import ctypes

import numpy as np
import pytest
import torch

from long_context_decode_02_b200 import synth
from tests import paged_reference as R


@pytest.fixture(scope="module")
def L():
    from long_context_decode_02_b200 import build
    build.build()
    from long_context_decode_02_b200 import lowram
    return lowram


def test_reference_codes_agree_with_the_type():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.TABLE, want, equal_nan=True)
    x = np.concatenate([np.random.default_rng(0).uniform(-448, 448, 20000),
                        2.0 ** np.random.default_rng(1).uniform(-12, 8, 20000),
                        [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 448.0, 1.0625, 1.1875, np.inf, np.nan]])
    x = x.astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(x), got)


@pytest.mark.parametrize("amax,want", [(0.0, 2.0 ** -64), (448.0, 1.0), (448.001, 2.0), (224.0, 0.5),
                                       (1e-30, 2.0 ** -64), (3.3e38, 2.0 ** 120)])
def test_reference_scale(amax, want):
    assert R.scale_for(amax) == want


def test_reference_append_is_independent_of_its_division():
    """Filling pages token by token, or at once, gives the same scales, and the same codes but
    for those that pass below 2^-6 (where e4m3 is subnormal)."""
    rng = np.random.default_rng(3)
    n, H, d, P = 41, 2, 64, 16
    k, v = rng.normal(size=(2, n, H, d)) * np.exp(rng.normal(size=(2, n, 1, 1)))
    empty = lambda: R.Pages(np.zeros((3, H, P, d), np.uint8), np.zeros((3, H, P, d), np.uint8),  # noqa: E731
                            np.ones((3, H)), np.ones((3, H)))
    once, steps = empty(), empty()
    once.append([[2, 0, 1]], [n], k, v, [n], [100], 1e4)
    for t in range(n):
        steps.append([[2, 0, 1]], [t + 1], k[t:t + 1], v[t:t + 1], [1], [100], 1e4)
    for name in "kv":
        assert np.array_equal(once.scale[name], steps.scale[name])
        a, b = R.decode(once.code[name]), R.decode(steps.code[name])
        same = a == b
        assert np.all(np.abs(a - b)[~same] <= 2.0 ** -9) and np.all(np.abs(a[~same]) < 2.0 ** -5)


def _cfg(L, **kw):
    return L.make_config(synth.CONFIGS[1], **kw)


def test_workspace_size(L):
    c = _cfg(L)
    assert L.paged_workspace_size(c, 1, 1) > 0
    assert L.paged_workspace_size(c, 64, 16) >= L.paged_workspace_size(c, 1, 1)
    n = ctypes.c_size_t()
    for seqs, nq, want in [(0, 1, L.ERR_SHAPE), (1, 0, L.ERR_SHAPE), (8193, 1, L.ERR_UNSUPPORTED),
                           (1, 17, L.ERR_UNSUPPORTED)]:
        assert L.lowram_paged_workspace_size(ctypes.byref(c), seqs, nq, ctypes.byref(n)) == want
    assert L.lowram_paged_workspace_size(ctypes.byref(c), 1, 1, None) == L.ERR_INVALID_ARG


def test_calls_without_a_context_are_refused(L):
    p = L.lowram_pages()
    assert L.lowram_paged_append(None, ctypes.byref(p), None, None, 0, 0, 0, None, 0, None, 1,
                                 None) == L.ERR_INVALID_ARG
    assert L.lowram_paged_attend(None, ctypes.byref(p), None, 1, None, None, None, 0,
                                 None) == L.ERR_INVALID_ARG
    assert L.lowram_paged_gather(None, ctypes.byref(p), None, 1, None, None,
                                 None) == L.ERR_INVALID_ARG


def _tensors(n_pages=4, H=2, P=16, d=64, seqs=2, width=3):
    return [torch.zeros(n_pages, H, P, d, dtype=torch.uint8),
            torch.zeros(n_pages, H, P, d, dtype=torch.uint8), torch.ones(n_pages, H),
            torch.ones(n_pages, H), torch.zeros(seqs, width, dtype=torch.int32),
            torch.zeros(seqs, dtype=torch.int32)]


def test_descriptor(L):
    p = L.paged_cache(*_tensors())
    assert (p.n_seqs, p.max_pages, p.n_pages, p.page_tokens) == (2, 3, 4, 16)
    t = _tensors()
    t[0] = t[0].view(torch.float8_e4m3fn)
    L.paged_cache(*t)


@pytest.mark.parametrize("at,make", [
    (0, lambda t: t[0][:, :, :8]),                     # shapes differ
    (1, lambda t: t[1].to(torch.int16)),
    (2, lambda t: t[2].double()),
    (3, lambda t: t[3][:, :1]),
    (4, lambda t: t[4].long()),
    (4, lambda t: t[4][0]),
    (5, lambda t: t[5][:1]),
    (1, lambda t: torch.zeros(4, 2, 64, 16, dtype=torch.uint8).transpose(2, 3)),   # strided
])
def test_descriptor_refusals(L, at, make):
    t = _tensors()
    t[at] = make(t)
    with pytest.raises(ValueError):
        L.paged_cache(*t)
