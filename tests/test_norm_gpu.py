"""mx_rmsnorm_quantize and mx_dequantize against 64 bits.

Tolerances.  h is one fp32 addition of values exact in fp32: 2^-24.  The sum of
squares is a chain of at most 64 terms a thread, 5 halvings and 32 warps: 101
roundings, with h's own error twice 103, and mean, eps and the root add three;
half of that reaches y, and three products more: y is within 2^-18 relative.  So each
scale is that of a block whose maximum is off by as much, and each code lies between
those of y (1 - 2^-18) and y (1 + 2^-18) under that scale (rounding is monotone)."""
import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _layer

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -18
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    mx.build()
    mx.lib()


def _check(q, x, r, w, eps, fmt, h_out):
    f64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    h, y = _layer.rmsnorm(f64(x), f64(r), f64(w), eps)
    rows, K = y.shape
    if r is not None:
        small = {F16: 2.0 ** -25}.get(r.dtype, 0.0)
        assert (np.abs(f64(h_out) - h) <= np.abs(h) * (HALF[r.dtype] + 2.0 ** -24) * (1 + 2.0 ** -8) + small).all()
    code = mx.scales_to_rowmajor(q.scales.cpu().numpy(), rows, K).astype(np.int64)
    amax = np.abs(y.reshape(rows, -1, 32)).max(2)
    assert ((code == _layer.scale_of(amax * (1 - TOL), fmt)) | (code == _layer.scale_of(amax * (1 + TOL), fmt))).all()
    unit = 2.0 ** (code - 127.0).repeat(32, 1)
    got = mx.mx_dequantize(q).double().cpu().numpy()
    a, b = _layer.nearest(y / unit * (1 - TOL), fmt) * unit, _layer.nearest(y / unit * (1 + TOL), fmt) * unit
    assert ((got >= np.minimum(a, b)) & (got <= np.maximum(a, b))).all()
    # rows and blocks that pad the last atoms
    plane = q.scales.cpu().numpy().reshape(-(-rows // 128), -(-K // 128), 32, 4, 4)
    full = plane.transpose(0, 3, 2, 1, 4).reshape(-(-rows // 128) * 128, -1)
    assert (full[rows:] == 0).all() and (full[:, K // 32:] == 0).all()


def _inputs(rows, K, xd, rd, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, K, generator=g, device="cuda") * torch.exp2(torch.randn(rows, 1, generator=g, device="cuda") * 2)
    r = None if rd is None else (torch.randn(rows, K, generator=g, device="cuda") * 5).to(rd)
    return x.to(xd), r, 1 + 0.3 * torch.randn(K, generator=g, device="cuda")


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (130, 96), (5, 160), (64, 1024), (33, 2080), (2, 8192), (700, 8192),
                                    (310, 5120), (3, 16384), (400, 16384), (2, 16416), (2, 32768)])
@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2, mx.E2M1])
@pytest.mark.parametrize("xd,rd", [(BF16, BF16), (F16, None), (F32, F16), (F32, F32), (BF16, F32), (F32, None)])
def test_against_64_bits(rows, K, fmt, xd, rd):
    x, r, w = _inputs(rows, K, xd, rd, rows + K)
    q, h = mx.mx_rmsnorm_quantize(x, w, fmt, residual=r, eps=1e-5)
    assert (h is None) == (r is None)
    _check(q, x, r, w, 1e-5, fmt, h)


@pytest.mark.parametrize("onto", ["residual", "x", "wide"])
def test_in_place_and_strided(onto):
    x, r, w = _inputs(37, 1056, BF16, BF16)
    wide = torch.full((37, 1200), 7.0, dtype=BF16, device="cuda")
    wide[:, 16:16 + 1056] = x
    xv = wide[:, 16:16 + 1056]
    x0, r0 = xv.clone(), r.clone()
    target = {"residual": r, "x": xv, "wide": torch.empty(37, 2000, dtype=BF16, device="cuda")[:, :1056]}[onto]
    q, h = mx.mx_rmsnorm_quantize(xv, w, mx.E4M3, residual=r, residual_out=target)
    assert h is target
    _check(q, x0, r0, w, 1e-6, mx.E4M3, h)
    assert (wide[:, :16] == 7).all() and (wide[:, 1072:] == 7).all()


def test_the_codes_are_those_of_mx_quantize():
    """One thread's order of additions apart, the same as norm and mx_quantize in turn: with a row
    of equal magnitudes y is exact in both."""
    x = torch.where(torch.rand(200, 512, device="cuda") < 0.5, -2.0, 2.0)
    w = torch.exp2(torch.randint(-3, 4, (512,), device="cuda").float())
    eps = 2.0 ** -70                             # nothing beside 4
    q, _ = mx.mx_rmsnorm_quantize(x.bfloat16(), w, mx.E4M3, eps=eps)
    ref = mx.mx_quantize(x / 2 * w, mx.E4M3)
    assert torch.equal(q.data, ref.data) and torch.equal(q.scales, ref.scales)


def test_rows_of_zeros_large_and_small_values():
    K = 1024
    x = torch.zeros(6, K, device="cuda")
    x[1] = 3.0e38                                # squares overflow
    x[2] = torch.randn(K, device="cuda") * 1e25
    x[3] = torch.randn(K, device="cuda") * 1e-25  # squares underflow: eps is all
    x[4, 5] = 1e30                               # one value beside zeros
    x[5] = torch.randn(K, device="cuda")
    w = torch.ones(K, device="cuda")
    for fmt in (mx.E4M3, mx.E5M2, mx.E2M1):
        q, _ = mx.mx_rmsnorm_quantize(x, w, fmt, eps=1e-6)
        _check(q, x, None, w, 1e-6, fmt, None)
        assert (mx.mx_dequantize(q)[0] == 0).all()


def test_small_values_in_rows_whose_squares_overflow():
    """y of what stands beside values of 2^64 and more is as exact as any: normal fp32 values under normal
    scales, however far below the row's largest (the bound's roundings and no other: factors of two are exact)."""
    K = 256
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(7, K, generator=g, device="cuda")
    x[0] *= 2.0 ** -30
    x[1] *= 2.0 ** -51
    x[2] *= torch.exp2(torch.arange(K, device="cuda") / 2 - 60)
    x[3] *= 2.0 ** 20
    x[4] *= 2.0 ** -58
    x[5] *= 2.0 ** 40
    x[6] *= 2.0 ** -20
    x[0, 0] = x[1, 77] = x[3, 200] = 2.0 ** 64
    x[2, 255] = x[5, 31] = 3.0e38
    x[4, 128] = x[6, 3] = 2.0 ** 66
    w = 1 + 0.3 * torch.randn(K, generator=g, device="cuda")
    w[64:96] *= 2.0 ** 30
    w[96:128] *= 2.0 ** -14
    for fmt in (mx.E4M3, mx.E5M2, mx.E2M1):
        q, _ = mx.mx_rmsnorm_quantize(x, w, fmt, eps=1e-6)
        _check(q, x, None, w, 1e-6, fmt, None)
        r = x.flip(1).contiguous()
        q, h = mx.mx_rmsnorm_quantize(x, w, fmt, residual=r, eps=1e-6)
        _check(q, x, r, w, 1e-6, fmt, h)


@pytest.mark.parametrize("rows,K", [(3, 64), (2, 4096), (3, 32768)])
def test_large_eps(rows, K):
    """eps counts whatever the squares do: mean squares of 4e34, whose sum overflows at 32768 values, beside an
    eps of the same size; and rows that a large eps divides down to 2^-90 and weights bring back."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(rows, K, generator=g, device="cuda") * 2e17
    w = 1 + 0.3 * torch.randn(K, generator=g, device="cuda")
    for eps in (1e34, 1e36, 3e38):
        q, _ = mx.mx_rmsnorm_quantize(x, w, mx.E4M3, eps=eps)
        _check(q, x, None, w, eps, mx.E4M3, None)
    small = x * 2.0 ** -140
    for up in (2.0 ** 60, 2.0 ** 100):
        q, _ = mx.mx_rmsnorm_quantize(small, w * up, mx.E5M2, eps=3e38)
        _check(q, small, None, w * up, 3e38, mx.E5M2, None)


def test_subnormal_values_under_huge_weights():
    """h f is sqrt(2) 2^-127, with 22 bits, and y sqrt(2) 2^-19 under a weight of 2^108: f w is beyond fp32, y is not."""
    x = torch.full((2, 64), 2.0 ** -22, device="cuda")
    x[:, 32:] = 2.0 ** -149
    x[1, ::2] *= -1
    w = torch.ones(64, device="cuda")
    w[32:] = 2.0 ** 108
    for fmt in (mx.E4M3, mx.E5M2, mx.E2M1):
        q, _ = mx.mx_rmsnorm_quantize(x, w, fmt, eps=1e-30)
        _check(q, x, None, w, 1e-30, fmt, None)


def test_nan_and_infinity_stay_in_their_rows():
    x = torch.randn(4, 256, device="cuda")
    x[1, 40], x[2, 100] = float("nan"), float("inf")
    w = torch.ones(256, device="cuda")
    q, _ = mx.mx_rmsnorm_quantize(x, w, mx.E4M3)
    v = mx.mx_dequantize(q)
    assert torch.isfinite(v[0]).all() and torch.isfinite(v[3]).all() and torch.isnan(v[1]).all()
    assert torch.isnan(v[2, 96:128]).all() and (v[2, :96] == 0).all() and (v[2, 128:] == 0).all()
    clean = x.clone()
    clean[1:3] = 1.0
    ref, _ = mx.mx_rmsnorm_quantize(clean, w, mx.E4M3)
    assert torch.equal(mx.mx_dequantize(ref)[[0, 3]], v[[0, 3]])


def test_it_feeds_the_product():
    """The A operand of mx_gemm: the same product as of the plane that mx_quantize makes of its
    values (which are exact in it)."""
    x, r, w = _inputs(77, 512, BF16, BF16)
    b = mx.mx_quantize(torch.randn(512, 256, device="cuda"), mx.E4M3, k_strided=True)
    q, _ = mx.mx_rmsnorm_quantize(x, w, mx.E4M3, residual=r)
    again = mx.mx_quantize(mx.mx_dequantize(q), mx.E4M3)
    assert torch.equal(mx.mx_dequantize(again), mx.mx_dequantize(q))
    assert torch.equal(mx.mx_gemm(q, b), mx.mx_gemm(again, b))
    assert mx.mx_last_error() == 0


def test_captured_on_a_side_stream_and_again():
    x, r, w = _inputs(256, 2048, BF16, BF16)
    want, h = mx.mx_rmsnorm_quantize(x, w, mx.E4M3, residual=r)
    out, ho = mx.empty_mx(mx.E4M3, 256, 2048), torch.empty_like(r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mx.mx_rmsnorm_quantize(x, w, mx.E4M3, residual=r, residual_out=ho, out=out)
    for _ in range(3):
        out.data.zero_(), out.scales.fill_(255), ho.zero_()
        graph.replay()
        assert torch.equal(out.data, want.data) and torch.equal(out.scales, want.scales) and torch.equal(ho, h)


# ------------------------------------------------------------------ values

@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2, mx.E2M1, mx.INT8, mx.INT4, mx.INT2])
@pytest.mark.parametrize("rows,K", [(1, 32), (130, 160), (257, 4096), (16, 96)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_values_of_every_code(fmt, rows, K, dtype):
    rng = np.random.default_rng(rows + K)
    q = mx.empty_mx(fmt, rows, K)
    q.data.copy_(torch.from_numpy(rng.integers(0, 256, q.data.numel()).astype(np.uint8)))
    scale = rng.integers(0, 256, q.scales.numel()).astype(np.uint8)
    if dtype != F32:
        scale = (120 + scale % 12).astype(np.uint8)
    scale[:1] = 255
    q.scales.copy_(torch.from_numpy(scale))
    raw = q.data.cpu().numpy()
    if fmt in (mx.E4M3, mx.E5M2, mx.INT8):
        from tests import _kv
        v = _kv.TABLES[fmt][raw].reshape(rows, K)
    else:
        n = 2 if fmt != mx.INT2 else 4
        bits = 8 // n
        c = np.stack([(raw >> (bits * i)) & (2 ** bits - 1) for i in range(n)], 1).reshape(rows, K).astype(np.int64)
        if fmt == mx.E2M1:
            v = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])[c]
        else:
            v = np.where(c >= 2 ** (bits - 1), c - 2 ** bits, c).astype(np.float64)
    code = mx.scales_to_rowmajor(scale, rows, K).astype(np.float64).repeat(32, 1)
    with np.errstate(over="ignore", invalid="ignore"):
        want = v * np.where(code == 255, np.nan, 2.0 ** (code - 127))
        want = torch.from_numpy(want.astype(np.float32)).to(dtype)   # (exact in fp32 but where it overflows)
    out = torch.empty(rows, K + 32, dtype=dtype, device="cuda")[:, 16:16 + K]
    got = mx.mx_dequantize(q, out_dtype=dtype, out=out).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0.0, 9e9, -9e9), want.nan_to_num(0.0, 9e9, -9e9))


def test_values_return_what_was_quantized():
    x = torch.randint(-6, 7, (300, 640), device="cuda").float() * 0.25
    x[:, ::32] = 1.75                            # every block's scale the same
    for fmt in (mx.E4M3, mx.INT8):
        assert torch.equal(mx.mx_dequantize(mx.mx_quantize(x, fmt)), x)


def test_operands_that_do_not_fit():
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    r = torch.randn(4, 64, device="cuda")
    for bad in (lambda: mx.mx_rmsnorm_quantize(x, w, mx.INT8), lambda: mx.mx_rmsnorm_quantize(x[:, :48], w[:48], mx.E4M3),
                lambda: mx.mx_rmsnorm_quantize(x, w, mx.E4M3, residual=r[:3]), lambda: mx.mx_rmsnorm_quantize(x, w, mx.E4M3, residual_out=r),
                lambda: mx.mx_rmsnorm_quantize(x, w, mx.E4M3, residual=r, residual_out=r.half()),
                lambda: mx.mx_rmsnorm_quantize(x, w, mx.E4M3, out=mx.empty_mx(mx.E5M2, 4, 64)),
                lambda: mx.mx_rmsnorm_quantize(x, w.cpu(), mx.E4M3), lambda: mx.mx_dequantize(mx.empty_mx(mx.E4M3, 4, 64), torch.float64)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(mx.MXError):
        mx.mx_rmsnorm_quantize(x, w, mx.E4M3, eps=0.0)
    with pytest.raises(mx.MXError):
        mx.mx_rmsnorm_quantize(torch.zeros(1, 32800, device="cuda"), torch.ones(32800, device="cuda"), mx.E4M3)


def test_no_rows_and_a_stream_argument():
    w = torch.ones(64, device="cuda")
    q, h = mx.mx_rmsnorm_quantize(torch.zeros(0, 64, device="cuda"), w, mx.E4M3, residual=torch.zeros(0, 64, device="cuda"))
    assert q.outer == 0 and h.shape == (0, 64) and mx.mx_dequantize(q).shape == (0, 64)
    x, r, w = _inputs(50, 512, F16, F16)
    want, hw = mx.mx_rmsnorm_quantize(x, w, mx.E5M2, residual=r)
    vw = mx.mx_dequantize(want, BF16)
    out, ho, vo = mx.empty_mx(mx.E5M2, 50, 512), torch.empty_like(r), torch.empty_like(vw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mx.mx_rmsnorm_quantize(x, w, mx.E5M2, residual=r, out=out, residual_out=ho, stream=side)
    mx.mx_dequantize(out, BF16, out=vo, stream=side)
    side.synchronize()
    assert torch.equal(out.data, want.data) and torch.equal(out.scales, want.scales) and torch.equal(ho, hw) and torch.equal(vo, vw)
