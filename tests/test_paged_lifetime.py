"""A paged cache's descriptor holds its tensors, and nothing holds the descriptor: dropping it
frees the pool at once, without the cyclic collector (which a full GPU does not start)."""
import gc
import weakref

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from long_context_decode_02_b200 import build
    build.build()
    from long_context_decode_02_b200 import lowram
    return lowram


def test_dropping_a_descriptor_frees_its_pool(L):
    t = [torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16, 64, dtype=torch.uint8),
         torch.ones(4, 2), torch.ones(4, 2), torch.zeros(2, 3, dtype=torch.int32),
         torch.zeros(2, dtype=torch.int32)]
    alive = [weakref.ref(x) for x in t]
    was = gc.isenabled()
    gc.disable()
    try:
        pages = L.paged_cache(*t)
        del t
        assert all(r() is not None for r in alive)
        # a call with it, refused for want of a context, leaves nothing behind either
        assert L.lowram_paged_attend(None, pages, None, 1, None, None, None, 0, None) == L.ERR_INVALID_ARG
        gone = weakref.ref(pages)
        del pages
        assert gone() is None and all(r() is None for r in alive)
    finally:
        if was:
            gc.enable()
