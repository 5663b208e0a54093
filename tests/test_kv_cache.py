"""The binding of the paged cache on the host: what a cache's C view says after
its planes changed, and what the calls refuse before the library."""
import copy
import os
import pickle
import subprocess
import sys

import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def _cache(pages=8, heads=2, page=16, d=64):
    return mx.KVCache(_u8(pages, heads, page, d), _u8(pages, heads, page, d), _u8(pages, heads),
                      _u8(pages, heads), mx.E4M3)


def _says(c):
    return c.pages, c.heads, c.page, c.d


def test_planes_of_another_geometry_at_the_same_address():
    """The bound on page ids and the tensor map come from the planes as they
    are at the call, not from the ones that stood at their address before."""
    cache = _cache()
    assert _says(cache.c()) == (8, 2, 16, 64)
    k, v, ks, vs = cache.k, cache.v, cache.k_scales, cache.v_scales
    cache.k, cache.v, cache.k_scales, cache.v_scales = k[:3], v[:3], ks[:3], vs[:3]
    assert cache.k.data_ptr() == k.data_ptr() and _says(cache.c()) == (3, 2, 16, 64)
    cache.k, cache.v = k.view(8, 2, 8, 128)[:3], v.view(8, 2, 8, 128)[:3]
    assert _says(cache.c()) == (3, 2, 8, 128)
    # in place, too
    cache = _cache()
    cache.c()
    for t, n in ((cache.k, (4, 2, 16, 64)), (cache.v, (4, 2, 16, 64)), (cache.k_scales, (4, 2)),
                 (cache.v_scales, (4, 2))):
        t.resize_(n)
    assert _says(cache.c()) == (4, 2, 16, 64)


@pytest.mark.parametrize("change", [
    lambda c: setattr(c, "v", c.v[:3]), lambda c: setattr(c, "k_scales", c.k_scales[:7]),
    lambda c: setattr(c, "v_scales", c.v_scales.view(4, 4)),
    lambda c: setattr(c, "k", c.k.as_strided((8, 2, 16, 64), (2048, 1024, 64, 0))),
    lambda c: setattr(c, "v_scales", c.v_scales.as_strided((8, 2), (0, 1)))])
def test_planes_that_no_longer_belong_together_are_refused(change):
    cache = _cache()
    cache.c()
    change(cache)
    with pytest.raises(ValueError):
        cache.c()


def test_a_cache_in_host_memory_is_refused():
    """Before anything else of the call is looked at: K, V and Q may well be
    on the GPU."""
    cache, q = _cache(), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="planes must be CUDA"):
        mx.mx_kv_append(cache, q, q, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="planes must be CUDA"):
        mx.mx_kv_attention(q, cache, i.view(3, 1), i[:2], i, 1)


def test_a_workspace_in_host_memory_is_refused():
    cache, q = _cache(), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="workspace"):
        mx.mx_kv_attention(q, cache, i.view(3, 1), i[:2], i, 1, workspace=_u8(1 << 20))


@pytest.mark.gpu
def test_a_workspace_that_holds_less_than_it_says_is_refused():
    mx.build()
    cache = mx.empty_kv_cache(mx.E4M3, 8, 2, 16, 64)
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    few = torch.zeros(16, dtype=torch.uint8, device="cuda")
    for ws in (few.expand(1 << 20, 16), few[::2], few.cpu()):
        with pytest.raises(ValueError, match="workspace"):
            mx.mx_kv_attention(q, cache, i.view(3, 1), i[:2], i, 1, workspace=ws)
    with pytest.raises(ValueError, match="planes must be CUDA"):
        mx.mx_kv_attention(q, _cache(), i.view(3, 1), i[:2], i, 1)
    with pytest.raises(ValueError, match="planes must be CUDA"):
        mx.mx_kv_append(_cache(), q, q, torch.zeros(2, dtype=torch.int64, device="cuda"))


def test_a_cache_can_be_copied():
    """deepcopy and pickle give a cache of its own planes."""
    cache = _cache()
    cache.k[3] = 7
    for other in (copy.deepcopy(cache), pickle.loads(pickle.dumps(cache))):
        assert torch.equal(other.k, cache.k) and other.fmt == cache.fmt
        c = other.c()
        assert c.k_data == other.k.data_ptr() != cache.k.data_ptr() and _says(c) == (8, 2, 16, 64)
    shallow = copy.copy(cache)
    shallow.k = cache.k.clone()
    assert cache.c().k_data == cache.k.data_ptr() and shallow.c().k_data == shallow.k.data_ptr()
