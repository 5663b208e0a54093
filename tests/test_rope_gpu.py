"""mx_rope against 64 bits, angles reduced with whole numbers.

Tolerances: the turn's fraction is rounded to fp32 (2^-24 of an angle of at most pi:
2^-22.3), sine and cosine are good to 2 units in 2^-24 and multiplied by the factor, two
products and a sum in fp32 (3 * 2^-24 of their sizes): in all less than 2^-20 of
|a| + |b|, times the factor; then the output's own rounding."""
import math

import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _layer

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    mx.build()
    mx.lib()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _check(got, x, pos, rope, neighbours=False, backward=False):
    rot = 2 * rope.freq.numel()
    x64 = x.double().cpu().numpy()
    want = _layer.rope(x64, pos, rope.freq.tolist(), rot, rope.factor, neighbours, backward)
    a = np.abs(x64[..., :rot])
    both = np.empty_like(a)
    if neighbours:
        both[..., ::2] = both[..., 1::2] = a[..., ::2] + a[..., 1::2]
    else:
        both[..., :rot // 2] = both[..., rot // 2:] = a[..., :rot // 2] + a[..., rot // 2:]
    bound = np.zeros_like(x64)
    bound[..., :rot] = both * abs(rope.factor) * 2.0 ** -20
    bound += np.abs(want) * HALF[x.dtype] * (1 + 2.0 ** -8) * (np.arange(x64.shape[2]) < rot)
    bound += 2.0 ** -25 * (np.arange(x64.shape[2]) < rot)      # f16's subnormal step
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("T,hq,hk,d,rot", [(1, 1, 1, 64, 64), (5, 32, 8, 128, 128), (3, 4, 0, 128, 32), (67, 6, 2, 72, 48),
                                           (40, 3, 1, 512, 512), (7, 2, 2, 1024, 16), (620, 4, 1, 64, 64), (1021, 5, 1, 24, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("neighbours", [False, True])
def test_positions_given(T, hq, hk, d, rot, dtype, neighbours):
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 2 ** 31, T) if T > 3 else np.array([0, 1, 2 ** 31 - 1])[:T]
    pos[-1:] = -17                               # a place in front of the first
    qkv = torch.randn(T, hq + 2 * hk, d, device="cuda").to(dtype)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk] if hk else None
    rope = mx.rope_frequencies(rot)
    for backward in (False, True):
        oq, ok = mx.mx_rope(q, k, rope, positions=_i32(pos), neighbours=neighbours, backward=backward)
        _check(oq, q, pos, rope, neighbours, backward)
        if hk:
            _check(ok, k, pos, rope, neighbours, backward)
        else:
            assert ok is None


@pytest.mark.parametrize("lens,new", [([9], [1]), ([5, 0, 7, 100], [5, 0, 2, 40]), ([33] * 33, [1] * 33),
                                      (list(range(40, 1300)), [i % 4 for i in range(1260)])])
def test_positions_of_a_plan(lens, new):
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + 6                          # rows behind the last request
    pos = np.concatenate([np.arange(n - z, n) for n, z in zip(lens, new)])
    q, k = torch.randn(T, 4, 64, device="cuda").bfloat16(), torch.randn(T, 2, 64, device="cuda").bfloat16()
    rope = mx.rope_frequencies(64, 500000.0, "parts", 8.0, 4096)
    oq, ok = torch.full_like(q, 3.0), torch.full_like(k, 3.0)
    mx.mx_rope(q, k, rope, lens=_i32(lens), cu=_i32(cu), out=(oq, ok))
    n = len(pos)
    _check(oq[:n], q[:n], pos, rope)
    _check(ok[:n], k[:n], pos, rope)
    assert (oq[n:] == 3).all() and (ok[n:] == 3).all()
    # in place: the same bits, and the rows behind as they were
    q2, k2 = q.clone(), k.clone()
    mx.mx_rope(q2, k2, rope, lens=_i32(lens), cu=_i32(cu), out=(q2, k2))
    assert torch.equal(q2[:n], oq[:n]) and torch.equal(q2[n:], q[n:]) and torch.equal(k2[:n], ok[:n]) and torch.equal(k2[n:], k[n:])


def test_tokens_in_front_of_the_first_request_and_no_request():
    q = torch.randn(8, 2, 64, device="cuda").bfloat16()
    rope = mx.rope_frequencies(64)
    out = torch.full_like(q, 3.0)
    mx.mx_rope(q, None, rope, lens=_i32([4]), cu=_i32([3, 5]), out=(out, None))
    _check(out[3:5], q[3:5], [2, 3], rope)
    assert (out[:3] == 3).all() and (out[5:] == 3).all()
    mx.mx_rope(q, None, rope, lens=_i32([]), cu=_i32([0]), out=(out, None))
    assert (out[:3] == 3).all()


def test_rest_of_the_head_in_place_of_a_projection():
    """Views of one projection, turned in place: the values' part and the heads' rest stay."""
    T, hq, hk, d = 50, 4, 2, 128
    qkv = torch.randn(T, hq + 2 * hk, d, device="cuda").half()
    before = qkv.clone()
    q, k, v = qkv.split([hq, hk, hk], 1)
    rope = mx.rope_frequencies(32)
    pos = np.arange(T) * 1000
    mx.mx_rope(q, k, rope, positions=_i32(pos), out=(q, k))
    _check(q, before[:, :hq], pos, rope)
    _check(k, before[:, hq:hq + hk], pos, rope)
    assert torch.equal(v, before[:, hq + hk:]) and torch.equal(qkv[..., 32:], before[..., 32:])


def test_gradient_is_the_transposed_map():
    """<rope(x), g> = <x, rope_backward(g)>, and against differences: the map is linear, so a step of
    any size gives its derivative, but for the rounding of the outputs (2^-11 each)."""
    T, d = 6, 64
    pos = _i32([0, 3, 77, 4000, 65537, 2 ** 30])
    rope = mx.Rope(mx.rope_frequencies(d).freq, 1.25)
    x, g = torch.randn(T, 3, d, device="cuda").half(), torch.randn(T, 3, d, device="cuda").half()
    y, _ = mx.mx_rope(x, None, rope, positions=pos)
    b, _ = mx.mx_rope(g, None, rope, positions=pos, backward=True)
    size = (x.double().abs() * b.double().abs()).sum() + (y.double().abs() * g.double().abs()).sum()
    assert abs((y.double() * g.double()).sum() - (x.double() * b.double()).sum()) <= 2.0 ** -10 * size
    for i in (0, 5, 31, 32, 63):
        e = torch.zeros_like(x)
        e[..., i] = 1.0
        up, _ = mx.mx_rope(e, None, rope, positions=pos)
        down, _ = mx.mx_rope(-e, None, rope, positions=pos)
        slope = ((up.double() - down.double()) / 2 * g.double()).sum(-1)
        assert ((slope - b[..., i].double()).abs() <= 2.0 ** -10 * ((up.double() * g.double()).abs().sum(-1) + b[..., i].double().abs()) + 2.0 ** -18).all()


@pytest.mark.parametrize("scaling,want", [
    ("linear", lambda f, i: f / 4), ("base", lambda f, i: (10000.0 * 4 ** (64 / 62)) ** (-2 * i / 64)),
    ("parts", lambda f, i: f * min(1, max(0, (8192 * f / (2 * math.pi) - 1) / 31)) + f / 4 * (1 - min(1, max(0, (8192 * f / (2 * math.pi) - 1) / 31))))])
def test_frequencies(scaling, want):
    rope = mx.rope_frequencies(64, scaling=scaling, factor=4.0, original=8192)
    for i, t in enumerate(rope.freq.tolist()):
        w = want(10000.0 ** (-2 * i / 64), i)
        assert abs(t * 2 * math.pi / 2.0 ** 64 - w) <= 1e-14 * w
    assert rope.factor == (1 + 0.1 * math.log(4) if scaling == "parts" else 1.0)


def test_captured():
    q = torch.randn(9, 4, 64, device="cuda").bfloat16()
    rope, lens, cu = mx.rope_frequencies(64), _i32([50]), _i32([0, 9])
    want, _ = mx.mx_rope(q, None, rope, lens=lens, cu=cu)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_rope(q, None, rope, lens=lens, cu=cu, out=(out, None))
    out.zero_()
    graph.replay()
    assert torch.equal(out, want)


def test_outputs_with_strides_and_a_stream_argument():
    T, pos = 70, np.arange(70) * 13
    q, k = torch.randn(T, 4, 64, device="cuda").half(), torch.randn(T, 2, 64, device="cuda").half()
    rope = mx.rope_frequencies(64)
    wide = torch.full((T, 3, 6, 72), 5.0, dtype=torch.float16, device="cuda")
    oq, ok = wide[:, 0, :4, :64], wide[:, 2, 1:3, 8:]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mx.mx_rope(q, k, rope, positions=_i32(pos), out=(oq, ok), stream=side)
    side.synchronize()
    _check(oq, q, pos, rope)
    _check(ok, k, pos, rope)
    assert (wide[:, 1] == 5).all() and (wide[:, 0, 4:] == 5).all() and (wide[:, 0, :4, 64:] == 5).all() and (wide[:, 2, 1:3, :8] == 5).all()


def test_operands_that_do_not_fit():
    q, rope = torch.randn(4, 2, 64, device="cuda").half(), mx.rope_frequencies(64)
    pos = _i32([0, 1, 2, 3])
    for bad in (lambda: mx.mx_rope(q, q.bfloat16(), rope, positions=pos), lambda: mx.mx_rope(q, q[:3], rope, positions=pos),
                lambda: mx.mx_rope(q, None, rope, positions=pos[:3]), lambda: mx.mx_rope(q, None, rope),
                lambda: mx.mx_rope(q, None, rope, positions=pos, out=(q, q)), lambda: mx.mx_rope(q, q, rope, positions=pos, out=(q, None)),
                lambda: mx.mx_rope(q.float(), None, rope, positions=pos), lambda: mx.mx_rope(q, None, rope, positions=pos.long())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(mx.MXError):              # more values than a head has
        mx.mx_rope(q, None, mx.rope_frequencies(128), positions=pos)
    with pytest.raises(mx.MXError):              # rows that lie on one another
        mx.mx_rope(q[:1].expand(4, 2, 64), None, rope, positions=pos)
