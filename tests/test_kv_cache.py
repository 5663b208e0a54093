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


def test_the_package_imports_without_torch_s_private_allocator():
    """The direct entry of the allocator is a saving, not a need."""
    code = ("import torch; del torch._C._dynamo.guards._empty_strided_cuda; "
            "import block_scaled_quantized_mx_gb300 as mx; print(len(mx.EXPORTS))")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, timeout=300)


class _On:
    """A tensor's device, as the choice of an allocator sees it."""

    def __init__(self, index):
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index


def test_outputs_are_made_where_the_operands_are(monkeypatch):
    """The direct entry knows the current device only and fills nothing."""
    made = []
    monkeypatch.setattr(mx, "_direct_empty", lambda *a: made.append(("direct",) + a))
    monkeypatch.setattr(torch, "empty_strided", lambda *a, **k: made.append((k["device"].index,) + a))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    make = lambda t: mx._allocator(t)((2, 3), (3, 1), torch.int32)  # noqa: E731
    make(_On(0))
    make(_On(1))
    monkeypatch.setattr(torch, "are_deterministic_algorithms_enabled", lambda: True)
    make(_On(0))
    monkeypatch.setattr(torch, "are_deterministic_algorithms_enabled", lambda: False)
    monkeypatch.setattr(mx, "_direct_empty", None)
    make(_On(0))
    assert [m[0] for m in made] == ["direct", 1, 0, 0] and all(m[1:3] == ((2, 3), (3, 1)) for m in made)


@pytest.mark.gpu
@pytest.mark.parametrize("direct", [True, False])
def test_outputs_of_each_allocator(direct, monkeypatch):
    mx.build()
    if not direct:
        monkeypatch.setattr(mx, "_direct_empty", None)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, stack = torch.full((2, 3), -1, **i32), torch.tensor([4, 3, 2, 1], **i32)
    lens, count = torch.tensor([0, 0], **i32), torch.tensor([4], **i32)
    plan = mx.mx_kv_extend(lens, torch.tensor([17, 3], **i32), table, stack, count, 16, 24)
    assert plan.lens.tolist() == [17, 3] and plan.cu.tolist() == [0, 17, 20] and plan.counts.tolist() == [1, 0]
    assert plan.slots.tolist() == [16 + i for i in range(16)] + [32, 48, 49, 50] + [-1] * 4
    cut = mx.mx_kv_truncate(plan.lens, torch.tensor([1, 0], **i32), table, stack, plan.counts, 16)
    assert cut.lens.tolist() == [1, 0] and cut.counts.tolist() == [3, 0]
    q = torch.ones(3, 2, 64, dtype=torch.float16, device="cuda")
    cache = mx.empty_kv_cache(mx.E4M3, 4, 2, 16, 64)
    args = (q, cache, table, torch.tensor([0, 0], **i32), torch.tensor([0, 1, 2], **i32), 1)
    o = mx.mx_kv_attention(*args, out_dtype=torch.float32)
    assert o.shape == (3, 2, 64) and o.is_contiguous() and o.dtype == torch.float32 and (o[:2] == 0).all()
    torch.use_deterministic_algorithms(True)
    try:                                         # rows of no request: as torch fills what nothing wrote
        assert mx.mx_kv_attention(*args)[2].isnan().all()
    finally:
        torch.use_deterministic_algorithms(False)


def test_the_workspace_s_size_is_asked_of_the_device_at_hand(monkeypatch):
    """It follows from the current device, and is 0 on one that the library
    does not run on: an answer for one is none for another."""
    answers = iter([0, 5, 9])

    class Lib:
        @staticmethod
        def mx_kv_attention_workspace_bytes(*a):
            return next(answers)

    monkeypatch.setattr(mx, "lib", lambda: Lib)
    assert [mx.kv_attention_workspace_bytes(24, 3, 64, 11) for _ in range(3)] == [0, 5, 9]
