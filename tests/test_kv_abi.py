"""The paged cache's calls without a GPU: refusals on the host before any
launch, the binding's checks, and the tests' own 64-bit restatement against
hand values."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _kv

X = 0x1000                                       # an address that is never followed
OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    mx.build()
    return mx.lib()


def _cache(**kw):
    a = dict(k_data=X, v_data=X, k_scales=X, v_scales=X, fmt=mx.E4M3, page=64, pages=4, heads=2,
             d=128)
    a.update(kw)
    return mx.CKVCache(*[a[n] for n, _ in mx.CKVCache._fields_])


BAD_CACHES = [(dict(fmt=mx.E2M1), INVALID), (dict(fmt=0), INVALID), (dict(page=8), SHAPE),
              (dict(page=48), SHAPE), (dict(page=256), SHAPE), (dict(d=96), SHAPE),
              (dict(d=256), SHAPE), (dict(heads=0), SHAPE), (dict(pages=0), SHAPE),
              (dict(pages=2 ** 25), SHAPE), (dict(k_data=None), INVALID),
              (dict(v_scales=None), INVALID), (dict(v_data=X + 8), ALIGN)]


def _append(L, cache=None, K=X, V=X, dtype=mx.DT_BF16, T=4, ks=(256, 128), vs=(256, 128), slots=X):
    c = cache or _cache()
    return L.mx_kv_append(ctypes.byref(c), K, V, dtype, T, *ks, *vs, slots, None)


def _attend(L, cache=None, Q=X, dtype=mx.DT_BF16, T=4, hq=8, qs=(1024, 128), table=X, stride=16,
            width=16, lens=X, cu=X, B=2, max_q=2, O=X, odt=mx.DT_BF16, os=(1024, 128), causal=1,
            window=0, scale=0.1, ws=None, n=0):
    c = cache or _cache()
    return L.mx_kv_attention(Q, dtype, T, hq, *qs, ctypes.byref(c), table, stride, width, lens, cu,
                             B, max_q, O, odt, *os, causal, window, scale, ws, n, None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_a_bad_cache_is_refused(L, kw, want):
    assert _append(L, _cache(**kw)) == want
    assert _attend(L, _cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=mx.DT_F32), INVALID), (dict(T=-1), SHAPE), (dict(K=None), INVALID),
    (dict(slots=None), INVALID), (dict(V=X + 4), ALIGN), (dict(ks=(252, 128)), SHAPE),
    (dict(vs=(256, 64)), SHAPE), (dict(vs=(64, 256)), SHAPE), (dict(T=0), OK)])
def test_append_refuses(L, kw, want):
    assert _append(L, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=mx.DT_F32), INVALID), (dict(odt=7), INVALID), (dict(hq=7), SHAPE),
    (dict(hq=0), SHAPE), (dict(causal=2), INVALID), (dict(window=-1), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(stride=8), SHAPE),
    (dict(width=0), SHAPE), (dict(B=-1), SHAPE), (dict(T=2 ** 30), SHAPE), (dict(Q=None), INVALID),
    (dict(table=None), INVALID), (dict(cu=None), INVALID), (dict(lens=None), INVALID),
    (dict(O=X + 8), ALIGN), (dict(qs=(1024, 100)), SHAPE), (dict(os=(64, 128)), SHAPE),
    (dict(ws=X + 4, n=1 << 20), ALIGN), (dict(max_q=-1), SHAPE), (dict(T=0), OK), (dict(B=0), OK)])
def test_attention_refuses(L, kw, want):
    assert _attend(L, **kw) == want


def test_workspace_bytes_refuses(L):
    f = L.mx_kv_attention_workspace_bytes
    for bad in ((8, 3, 128, 1), (8, 0, 128, 1), (0, 1, 128, 1), (8, 2, 80, 1), (8, 2, 128, 0)):
        assert f(*bad) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(B=16385), SHAPE), (dict(page=24), SHAPE), (dict(width=0), SHAPE),
    (dict(stride=2), SHAPE), (dict(size=-1), SHAPE), (dict(lens=None), INVALID),
    (dict(change=None), INVALID), (dict(table=None), INVALID), (dict(stack=None), INVALID),
    (dict(count=None), INVALID), (dict(lens_out=None), INVALID), (dict(counts=None), INVALID)])
def test_page_calls_refuse(L, kw, want):
    a = dict(B=2, page=16, width=4, stride=4, size=8, lens=X, change=X, table=X, stack=X, count=X,
             lens_out=X, counts=X)
    a.update(kw)
    assert L.mx_kv_extend(a["lens"], a["change"], a["B"], a["table"], a["stride"], a["width"],
                          a["stack"], a["size"], a["count"], a["page"], a["lens_out"], X, X, 32,
                          a["counts"], None) == want
    assert L.mx_kv_truncate(a["lens"], a["change"], a["B"], a["table"], a["stride"], a["width"],
                            a["stack"], a["size"], a["count"], a["page"], a["lens_out"],
                            a["counts"], None) == want


def test_extend_refuses_its_slots(L):
    assert L.mx_kv_extend(X, X, 2, X, 4, 4, X, 8, X, 16, X, X, None, 4, X, None) == INVALID
    assert L.mx_kv_extend(X, X, 2, X, 4, 4, X, 8, X, 16, X, X, X, -1, X, None) == SHAPE


def test_binding_refuses_before_the_library():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    cache = mx.KVCache(u8(4, 2, 16, 64), u8(4, 2, 16, 64), u8(4, 2), u8(4, 2), mx.E4M3)
    with pytest.raises(ValueError):
        mx.KVCache(u8(4, 2, 16, 64), u8(4, 2, 32, 64), u8(4, 2), u8(4, 2), mx.E4M3)
    with pytest.raises(ValueError):
        mx.KVCache(u8(4, 2, 16, 64), u8(4, 2, 16, 64), u8(2, 4), u8(4, 2), mx.E4M3)
    with pytest.raises(ValueError):
        mx.KVCache(u8(4, 2, 16, 64).float(), u8(4, 2, 16, 64), u8(4, 2), u8(4, 2), mx.E4M3)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):              # not on the GPU
        mx.mx_kv_extend(i, i, i.view(2, 1), i, i, 16, 4)
    with pytest.raises(ValueError):
        mx.mx_kv_truncate(i, i, i.view(2, 1), i, i, 16)
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mx.mx_kv_append(cache, q, q, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        mx.mx_kv_attention(q, cache, i.view(2, 1), i, i, 1)


# ------------------------------------------------------------------ the restatement itself

def test_codes_and_rounding_by_hand():
    t = _kv.TABLES
    assert t[_kv.E4M3][0x7E] == 448 and t[_kv.E4M3][0x01] == 2.0 ** -9 and math.isnan(t[_kv.E4M3][0x7F])
    assert t[_kv.E5M2][0x7B] == 57344 and t[_kv.E5M2][0x01] == 2.0 ** -16 and t[_kv.INT8][0xFF] == -1
    # ties to the even code, saturation, signed zero
    assert list(_kv.encode([17.0, 19.0, 1e9, -1e9, -0.0, 2.0 ** -10, 3 * 2.0 ** -10], _kv.E4M3)) == \
        [0x58, 0x5A, 0x7E, 0xFE, 0x80, 0x00, 0x02]
    assert list(_kv.encode([0.5, 1.5, -0.5, 127.5, -200], _kv.INT8)) == [0, 2, 0, 127, 128]
    ref = torch.arange(-600, 600, dtype=torch.float64) / 1.7
    got = _kv.encode(ref.numpy(), _kv.E4M3)
    want = ref.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (got == want).all()
    assert _kv.scale_code(448.0, _kv.E4M3) == 127 and _kv.scale_code(0.0, _kv.INT8) == 0
    assert _kv.scale_code(500.0, _kv.E4M3) == 127 and _kv.scale_code(512.0, _kv.E4M3) == 128


def test_append_restatement_by_hand():
    k = np.zeros((1, 1, 16, 64), np.uint8)
    ks = np.zeros((1, 1), np.uint8)
    v, vs = k.copy(), ks.copy()
    K = np.full((1, 1, 64), 100.0)
    _kv.append(k, v, ks, vs, _kv.INT8, K, K, [0])
    assert ks[0, 0] == 127 and (k[0, 0, 0] == 100).all()
    _kv.append(k, v, ks, vs, _kv.INT8, K * 4.02, K, [1])   # the scale grows by 4
    assert ks[0, 0] == 129 and (k[0, 0, 0] == 25).all() and (k[0, 0, 1] == 100).all()   # 402 / 4 = 100.5: even
    assert vs[0, 0] == 127 and (v[0, 0, :2] == 100).all()


def test_attention_restatement_by_hand():
    # two keys with equal scores: the mean of the values; a row before all keys: 0
    k = np.zeros((2, 1, 16, 64), np.uint8)
    v = k.copy()
    v[1, 0, 0], v[1, 0, 1] = 2, 6
    s = np.full((2, 1), 127, np.uint8)
    Q = np.ones((3, 1, 64))
    o, *_ = _kv.attention(Q, k, v, s, s, _kv.INT8, np.array([[1]]), [2], [0, 3], 1.0)
    assert (o[0] == 0).all() and (o[1] == 2).all() and (o[2] == 4).all()


def test_extend_and_truncate_restatement_by_hand():
    table = np.full((2, 3), -1, np.int32)
    out = _kv.extend([0, 0], [17, 3], table, [9, 8, 7, 6], 4, 16, 24)
    assert out == ([17, 20 - 17], [0, 17, 20], [96 + i for i in range(16)] + [112] +
                   [128, 129, 130] + [-1] * 4, [1, 0])
    stack = [9, -1, -1, -1]
    assert _kv.truncate([17, 3], [1, 0], table, stack, 1, 16) == ([1, 0], [3, 0])
    assert stack == [9, 8, 7, -1] and table.tolist() == [[6, -1, -1], [-1, -1, -1]]
