"""The calls for shared pages without a GPU: refusals on the host before any
launch, the binding's checks, and the tests' restatement against hand values."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _share

X = 0x1000                                       # an address that is never followed
OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    mx.build()
    return mx.lib()


def _cache(**kw):
    a = dict(k_data=X, v_data=X, k_scales=X, v_scales=X, fmt=mx.E4M3, page=64, pages=4, heads=2, d=128)
    a.update(kw)
    return mx.CKVCache(*[a[n] for n, _ in mx.CKVCache._fields_])


SIZES = [(dict(B=-1), SHAPE), (dict(B=16385), SHAPE), (dict(width=0), SHAPE), (dict(stride=2), SHAPE),
         (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(refs=None), INVALID), (dict(counts=None), INVALID),
         (dict(out=None), INVALID)]
STACK = [(dict(size=-1), SHAPE), (dict(stack=None), INVALID), (dict(count=None), INVALID), (dict(change=None), INVALID)]
PAGES = [(dict(page=24), SHAPE), (dict(pages=0), SHAPE), (dict(pages=2 ** 28), SHAPE)]


def _args(kw):
    a = dict(B=2, page=16, width=4, stride=4, size=8, lens=X, change=X, table=X, stack=X, count=X, out=X, counts=X, refs=X,
             pages=8, src=X, dst=X, forks=2, copies=X, cache={})
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,want", SIZES + STACK + PAGES)
def test_release_refuses(L, kw, want):
    a = _args(kw)
    assert L.mx_kv_release(a["lens"], a["change"], a["B"], a["table"], a["stride"], a["width"], a["stack"], a["size"], a["count"],
                           a["refs"], a["pages"], a["page"], a["out"], a["counts"], None) == want


@pytest.mark.parametrize("kw,want", SIZES + PAGES + [
    (dict(forks=-1), SHAPE), (dict(forks=16385), SHAPE), (dict(src=None), INVALID), (dict(dst=None), INVALID),
    (dict(change=None), INVALID)])
def test_fork_refuses(L, kw, want):
    a = _args(kw)
    assert L.mx_kv_fork(a["lens"], a["B"], a["src"], a["dst"], a["change"], a["forks"], a["table"], a["stride"], a["width"],
                        a["refs"], a["pages"], a["page"], a["out"], a["counts"], None) == want


@pytest.mark.parametrize("kw,want", SIZES + STACK + [
    (dict(copies=None), INVALID), (dict(cache=dict(page=24)), SHAPE), (dict(cache=dict(fmt=mx.E2M1)), INVALID),
    (dict(cache=dict(k_data=None)), INVALID), (dict(cache=dict(v_data=X + 8)), ALIGN)])
def test_own_refuses(L, kw, want):
    a = _args(kw)
    c = _cache(**a["cache"])
    assert L.mx_kv_own(ctypes.byref(c), a["lens"], a["change"], a["B"], a["table"], a["stride"], a["width"], a["stack"], a["size"],
                       a["count"], a["refs"], a["out"], a["copies"], a["counts"], None) == want


def test_binding_refuses_before_the_library():
    i = torch.zeros(2, dtype=torch.int32)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    cache = mx.KVCache(u8(4, 2, 16, 64), u8(4, 2, 16, 64), u8(4, 2), u8(4, 2), mx.E4M3)
    for bad in (lambda: mx.mx_kv_fork(i, i, i, i, i.view(2, 1), i, 16), lambda: mx.mx_kv_release(i, i, i.view(2, 1), i, i, i, 16),
                lambda: mx.mx_kv_own(cache, i, i, i.view(2, 1), i, i, i)):
        with pytest.raises(ValueError):
            bad()


def test_restatement_by_hand():
    table, refs = np.full((3, 2), -1, np.int32), [0] * 4
    table[0] = [3, 1]
    assert _share.fork([20, 0, 0], [0, 0, 0], [1, 2, 2], [20, 17, 16], table, refs, 16) == ([20, 20, 17], [1])
    assert refs == [0, 2, 0, 2] and table.tolist() == [[3, 1]] * 3
    # 0 and 1 write, 2 does not: both get copies, and 2 holds the page alone
    assert _share.own([20, 20, 17], [1, 1, 0], table, [0, 2], 2, refs, 16) == \
        ([1, 1, 0], [[1, 2, 4], [1, 0, 4], [-1] * 3], [0, 0])
    assert refs == [0, 0, 0, 2] and table.tolist() == [[3, 2], [3, 0], [3, 1]]
    stack = [0, 2, -1, -1]
    assert _share.release([20, 20, 17], [0, 16, 0], table, stack, 0, refs, 16) == ([0, 16, 0], [3, 0])
    # freed: 2 by request 0, 0 by request 1, 1 by request 2
    assert stack == [1, 0, 2, -1] and refs == [0, 0, 0, 0]


def _shared(L, **kw):
    a = dict(cache={}, Q=X, dtype=mx.DT_BF16, T=4, hq=8, qs=(1024, 128), table=X, stride=16, width=16, lens=X, cu=X, B=2, max_q=2,
             groups=X, shared=X, n=1, O=X, odt=mx.DT_BF16, os=(1024, 128), causal=1, scale=0.1, ws=None, bytes=0)
    a.update(kw)
    c = _cache(**a["cache"])
    return L.mx_kv_attention_shared(a["Q"], a["dtype"], a["T"], a["hq"], *a["qs"], ctypes.byref(c), a["table"], a["stride"], a["width"],
                                    a["lens"], a["cu"], a["B"], a["max_q"], a["groups"], a["shared"], a["n"], a["O"], a["odt"],
                                    *a["os"], a["causal"], a["scale"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(cache=dict(fmt=mx.E2M1)), INVALID), (dict(cache=dict(d=96)), SHAPE), (dict(cache=dict(k_data=X + 8)), ALIGN),
    (dict(dtype=mx.DT_F32), INVALID), (dict(odt=7), INVALID), (dict(hq=7), SHAPE), (dict(hq=0), SHAPE), (dict(causal=2), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(stride=8), SHAPE), (dict(width=0), SHAPE), (dict(B=-1), SHAPE), (dict(B=16385), SHAPE),
    (dict(n=-1), SHAPE), (dict(n=16385), SHAPE), (dict(T=2 ** 29), SHAPE), (dict(groups=None), INVALID), (dict(shared=None), INVALID),
    (dict(Q=None), INVALID), (dict(table=None), INVALID), (dict(cu=None), INVALID), (dict(lens=None), INVALID),
    (dict(O=X + 8), ALIGN), (dict(qs=(1024, 100)), SHAPE), (dict(ws=X + 4, bytes=1 << 30), ALIGN), (dict(max_q=-1), SHAPE),
    (dict(T=0), OK), (dict(B=0), OK)])
def test_shared_attention_refuses(L, kw, want):
    assert _shared(L, **kw) == want


def test_shared_workspace_bytes_refuses(L):
    f = L.mx_kv_attention_shared_workspace_bytes
    for bad in ((4, 8, 3, 128, 1, 2, 1), (4, 8, 0, 128, 1, 2, 1), (4, 0, 1, 128, 1, 2, 1), (4, 8, 2, 80, 1, 2, 1),
                (4, 8, 2, 128, 0, 2, 1), (0, 8, 2, 128, 1, 2, 1), (4, 8, 2, 128, 1, 0, 1), (4, 8, 2, 128, 1, 2, 0),
                (4, 8, 2, 128, 1, 16385, 1), (4, 8, 2, 128, 1, 2, 16385), (2 ** 28, 8, 2, 128, 1, 2, 1)):
        assert f(*bad) == 0


def test_the_binding_of_shared_attention_refuses():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    cache = mx.KVCache(u8(4, 2, 16, 64), u8(4, 2, 16, 64), u8(4, 2), u8(4, 2), mx.E4M3)
    i, q = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mx.mx_kv_attention_shared(q, cache, i.view(2, 1), i, i, 1, i, i)
