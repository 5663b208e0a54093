"""mx_rmsnorm_quantize, mx_dequantize and mx_rope without a GPU: refusals on
the host before any launch, the binding's checks, and the tests' restatement
against hand values."""
import ctypes
import decimal
import math

import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _layer

X = 0x1000                                       # an address that is never followed
OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    mx.build()
    return mx.lib()


def _tensor(**kw):
    a = dict(data=X, scales=X, fmt=mx.E4M3, outer=4, K=256)
    a.update(kw)
    return mx.CMXTensor(*[a[n] for n in ("data", "scales", "fmt", "outer", "K")])


@pytest.mark.parametrize("kw,want", [
    (dict(out=dict(fmt=mx.INT8)), INVALID), (dict(out=dict(fmt=9)), INVALID), (dict(out=dict(K=40)), SHAPE),
    (dict(out=dict(K=32800)), SHAPE), (dict(out=dict(data=X + 8)), ALIGN), (dict(xdt=3), INVALID), (dict(rdt=-1), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID), (dict(eps=-1.0), INVALID),
    (dict(w=None), INVALID), (dict(w=X + 4), ALIGN), (dict(x=None), INVALID), (dict(x=X + 2), ALIGN), (dict(ldx=248), SHAPE),
    (dict(ldx=260), SHAPE), (dict(r=None), INVALID), (dict(o=None), INVALID), (dict(ldr=100), SHAPE), (dict(ldo=0), SHAPE),
    (dict(o=X + 8), ALIGN), (dict(out=dict(outer=0)), OK), (dict(out=dict(K=0)), OK)])
def test_norm_refuses(L, kw, want):
    a = dict(x=X, xdt=mx.DT_BF16, ldx=256, r=X, rdt=mx.DT_F32, ldr=256, w=X, eps=1e-6, o=X, ldo=256, out={})
    a.update(kw)
    out = _tensor(**a["out"])
    assert L.mx_rmsnorm_quantize(a["x"], a["xdt"], a["ldx"], a["r"], a["rdt"], a["ldr"], a["w"], a["eps"], a["o"], a["ldo"],
                                 ctypes.byref(out), None) == want


def test_norm_refuses_without_a_tensor(L):
    assert L.mx_rmsnorm_quantize(X, 1, 256, None, 0, 0, X, 1e-6, None, 0, None, None) == INVALID


@pytest.mark.parametrize("kw,dtype,ld,want", [
    (dict(fmt=0), 0, 256, INVALID), ({}, 5, 256, INVALID), ({}, 0, 252, SHAPE), ({}, 1, 260, SHAPE), ({}, 0, 2 ** 31, SHAPE),
    (dict(scales=None), 0, 256, INVALID), (dict(outer=0), 0, 256, OK)])
def test_values_refuse(L, kw, dtype, ld, want):
    a = _tensor(**kw)
    assert L.mx_dequantize(ctypes.byref(a), X, dtype, ld, None) == want
    assert L.mx_dequantize(None, X, dtype, ld, None) == INVALID


def _rope(L, a={}, b=None, dtype=mx.DT_BF16, T=4, d=128, freq=X, rot=128, factor=1.0, pos=X, lens=None, cu=None, B=0, nb=0, bw=0):
    def operand(kw):
        o = dict(x=X, y=X, heads=8, xt=1024, xh=128, yt=1024, yh=128)
        o.update(kw)
        return mx.CRopeOperand(*o.values())
    first = ctypes.byref(operand(a)) if a is not None else None
    return L.mx_rope(first, None if b is None else ctypes.byref(operand(b)), dtype, T, d, freq, rot, factor, pos, lens, cu, B,
                     nb, bw, None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=None), INVALID), (dict(dtype=mx.DT_F32), INVALID), (dict(nb=2), INVALID), (dict(bw=-1), INVALID),
    (dict(factor=math.nan), INVALID), (dict(factor=math.inf), INVALID), (dict(d=132), SHAPE), (dict(d=1032), SHAPE),
    (dict(d=8, rot=8), SHAPE), (dict(rot=24), SHAPE), (dict(rot=144), SHAPE), (dict(rot=0), SHAPE), (dict(d=1024, rot=528), SHAPE),
    (dict(T=-1), SHAPE), (dict(B=-1), SHAPE), (dict(a=dict(heads=0)), SHAPE), (dict(b=dict(heads=65536)), SHAPE),
    (dict(a=dict(xh=64)), SHAPE), (dict(b=dict(yt=100)), SHAPE), (dict(a=dict(x=None)), INVALID), (dict(b=dict(y=None)), INVALID),
    (dict(b=dict(x=X + 8)), ALIGN), (dict(freq=None), INVALID), (dict(pos=None, B=2, lens=X), INVALID),
    (dict(pos=None, B=2, cu=X), INVALID), (dict(pos=None), OK), (dict(T=0), OK)])
def test_rope_refuses(L, kw, want):
    assert _rope(L, **kw) == want


def test_binding_refuses_before_the_library():
    x, w = torch.zeros(4, 64), torch.ones(64)
    for bad in (lambda: mx.mx_rmsnorm_quantize(x, w, mx.E4M3),                       # not on the GPU
                lambda: mx.mx_rmsnorm_quantize(x.double(), w, mx.E4M3),
                lambda: mx.mx_rmsnorm_quantize(x, w.half(), mx.E4M3),
                lambda: mx.mx_rmsnorm_quantize(x, w[:32], mx.E4M3),
                lambda: mx.mx_rmsnorm_quantize(x.t(), torch.ones(4), mx.E4M3),
                lambda: mx.mx_rope(x.view(4, 1, 64).half(), None, mx.rope_frequencies(64, device="cpu")),
                lambda: mx.rope_frequencies(24), lambda: mx.rope_frequencies(64, factor=0.5),
                lambda: mx.rope_frequencies(64, factor=2.0), lambda: mx.rope_frequencies(64, scaling="none"),
                lambda: mx.rope_frequencies(64, base=1.0)):
        with pytest.raises(ValueError):
            bad()


def test_frequencies_by_hand():
    f = mx.rope_frequencies(16, 10000.0, device="cpu")
    assert f.factor == 1.0 and f.freq[0].item() == round(2.0 ** 64 / (2 * math.pi)) and f.freq.numel() == 8
    g = mx.rope_frequencies(16, 10000.0, "linear", 4.0, device="cpu")
    assert all(abs(4 * b - a) <= 4096 for a, b in zip(f.freq.tolist(), g.freq.tolist()))


def _quarter_turns(bits):
    """pi / 4 times 2^bits, by Machin's formula in whole numbers."""
    def arctan(n):
        term, total, k = (1 << (bits + 40)) // n, 0, 0
        while term:
            total += (-1) ** k * term // (2 * k + 1)
            term, k = term // (n * n), k + 1
        return total
    return (4 * arctan(5) - arctan(239)) >> 40


@pytest.mark.parametrize("rot,base,scaling,factor", [
    (16, 10000.0, "parts", 1.0), (64, 10000.0, "linear", 8.0), (128, 500000.0, "linear", 3.0), (256, 2.0, "linear", 1.0),
    (16, 10000.0, "base", 128.0), (64, 500000.0, "parts", 8.0), (128, 10000.0, "parts", 4.0)])
def test_frequencies_against_roots(rot, base, scaling, factor):
    """Powers of base^(-2 / rot) as repeated square roots, in 60 digits.  The library's are doubles: of
    x = base^(-2 i / rot) the exponent's rounding costs ln(1 / x) 2^-53 of itself, the power two and the base (raised)
    one, a scaling three at most, 2 pi and the division two.  x (8 + ln(1 / x)) is 8 at most: 8 / 2 pi 2^-53 turns, less
    than 2^-52."""
    D, before = decimal.Decimal, decimal.getcontext().prec
    decimal.getcontext().prec = 60
    two_pi = D(8 * _quarter_turns(200)) / (1 << 200)
    b = D(base)
    if scaling == "base":                        # 128^(16 / 14) = 2^8
        b *= 256
    step, k = b, rot // 2
    while k > 1:
        step, k = step.sqrt(), k // 2
    want = [step ** -i for i in range(rot // 2)]
    if scaling == "linear":
        want = [x / D(factor) for x in want]
    if scaling == "parts":
        keep = [min(D(1), max(D(0), (8192 * x / two_pi - 1) / 31)) for x in want]
        want = [x * a + x / D(factor) * (1 - a) for x, a in zip(want, keep)]
    got = mx.rope_frequencies(rot, base, scaling, factor, original=8192, device="cpu").freq.tolist()
    off = [abs(D(g) - x / two_pi * 2 ** 64) for g, x in zip(got, want)]
    decimal.getcontext().prec = before
    assert len(got) == rot // 2 and max(off) <= 2 ** 12


def test_restatement_by_hand():
    assert list(_layer.nearest(np.array([5.0, 2.5, 0.25, 0.75, 7.0, -1.25]), _layer.E2M1)) == [4.0, 2.0, 0.0, 1.0, 6.0, -1.0]
    assert list(_layer.nearest(np.array([17.0, 19.0, 1e9, 2.0 ** -10]), _layer.E4M3)) == [16.0, 20.0, 448.0, 0.0]
    h, y = _layer.rmsnorm(np.array([[3.0, 4.0]]), None, np.array([1.0, 2.0]), 0.0)
    assert np.allclose(y, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]])
    # a quarter turn each position: (1, 0) -> (0, 1) -> (-1, 0)
    x = np.tile([1.0, 0.0], (3, 1, 1))
    assert np.allclose(_layer.rope(x, [0, 1, 2], [1 << 62], 2)[:, 0], [[1, 0], [0, 1], [-1, 0]])


def test_packed_structs_are_the_c_structs():
    a = mx.CRopeOperand(1, 2, 3, 4, 5, 6, 7)
    assert bytes(a) == mx._rope_struct(1, 2, 3, 4, 5, 6, 7)
    t = mx.CMXTensor(1, 2, 3, 4, 5)
    assert bytes(t) == mx._mx_struct(1, 2, 3, 4, 5)
