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
