"""The operators around the cache's attention in one run, as a server makes it:
prompts, samples forked from them, copies of the pages that they write, rotary
positions, the attention over what they share, and what they give back; each step
against 64 bits over what the cache then holds."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _kv, _layer

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve.py")


@pytest.fixture(scope="module")
def serve():
    mx.build()
    spec = importlib.util.spec_from_file_location("serve", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    mx.set_shared_bytes(0)                       # short prefixes are shared too
    yield m
    mx.set_shared_bytes(-1)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _sound(s, lens):
    """Every page is free, or held by one request more than refs says."""
    held = np.zeros(s.refs.numel(), int)
    table = s.table.cpu().numpy()
    for b, n in enumerate(lens):
        np.add.at(held, table[b, :-(-n // s.page)], 1)
    free = s.stack[:s.counts[0].item()].tolist()
    assert len(set(free)) == len(free) and (held[free] == 0).all() and len(free) + (held > 0).sum() == len(held)
    assert (np.maximum(held - 1, 0) == s.refs.cpu().numpy()).all()


@pytest.mark.parametrize("fmt,page", [(mx.E4M3, 16), (mx.INT8, 32)])
def test_samples_of_two_prompts(serve, fmt, page):
    layer = serve.Layer(256, 6, 2, 64)
    B = 9                                        # prompts in 0 and 5, samples behind them
    s = serve.Server(layer, requests=B, pages=80, page=page, longest=256, most_new=128, fmt=fmt)
    groups = _i32([0, 5, 9])
    lens = [0] * B
    fork = ([0, 0, 0, 0, 5, 5, 5], [1, 2, 3, 4, 6, 7, 8], [117, 117, 100, 117, 61, 61, 0])
    steps = [  # keep, new, fork, in groups
        ([0] * B, [117, 0, 0, 0, 0, 61, 0, 0, 0], None, False),
        ([117, 0, 0, 0, 0, 61, 0, 0, 0], [1, 1, 1, 1, 1, 0, 1, 1, 3], fork, True),
        (None, [1, 4, 1, 1, 2, 1, 1, 1, 1], None, True),                     # drafts
        ([119, 119, 0, 119, 50, 62, 0, 30, 4], [1, 1, 0, 2, 1, 1, 0, 1, 1], None, True),   # dropped; ended
        (None, [1] * B, ([0, 7], [2, 6], [64, 31]), True),                   # forked anew
        ([0] * B, [3] + [0] * 8, None, False)]
    for keep, new, forks, grouped in steps:
        keep = list(lens) if keep is None else keep
        now = [min(k, n) for k, n in zip(keep, lens)]
        if forks:
            for a, b, n in zip(*forks):
                now[b] = min(n, now[a])
        x = torch.randn(sum(new), 256, device="cuda").bfloat16()
        y, q, o, plan = s.step(_i32(keep), _i32(new), x, max(new), fork=[_i32(f) for f in forks] if forks else None,
                               groups=groups if grouped else None)
        lens = [k + n for k, n in zip(now, new)]
        assert plan.lens.tolist() == lens and plan.counts.tolist()[1] == 0 and torch.isfinite(y).all()
        _sound(s, lens)
        c = s.cache
        planes = [t.cpu().numpy() for t in (c.k, c.v, c.k_scales, c.v_scales)]
        e = _kv.attention(q.double().cpu().numpy(), *planes, fmt, s.table.cpu().numpy(), lens, plan.cu.tolist(), 64 ** -0.5)
        err = np.abs(o.double().cpu().numpy() - e[0])
        assert (err <= _kv.bound(*e, torch.bfloat16)).all()
        # queries: the projection of the norm's MX tensor, turned to the plan's positions.  bf16 before
        # and after the turn: half a step of 2^-8 of each, and the turn of what the first left
        # (another product of the same codes differs in fp32's last bits, a step of bf16 at the most)
        a, _ = mx.mx_rmsnorm_quantize(x, layer.norm, mx.E4M3)
        raw = (mx.mx_dequantize(a).double() @ mx.mx_dequantize(layer.w_qkv).double().t()).view(len(x), 10, 64)[:, :6].cpu().numpy()
        pos = np.concatenate([np.arange(n - z, n) for n, z in zip(lens, new)])
        want = _layer.rope(raw, pos, layer.rope.freq.tolist(), 64)
        both = np.abs(raw[..., :32]) + np.abs(raw[..., 32:])
        tol = np.concatenate([both, both], -1) * (2.0 ** -8 + 2.0 ** -15) + np.abs(want) * 2.0 ** -8 + 2.0 ** -14
        assert (np.abs(q.double().cpu().numpy() - want) <= tol).all()
    assert s.counts.tolist()[0] == 80 - 1 and s.refs.sum().item() == 0
    assert mx.mx_last_error() == 0


def test_samples_that_say_the_same_hear_the_same(serve):
    """Samples of one prompt with the same tokens: the same rows, bit for bit, as each would have
    alone (the rows of a unit are summed alike)."""
    layer = serve.Layer(256, 4, 1, 128)
    s = serve.Server(layer, requests=4, pages=40, page=16, longest=256, most_new=128)
    x = torch.randn(90, 256, device="cuda").bfloat16()
    s.step(_i32([0] * 4), _i32([90, 0, 0, 0]), x, 90)
    one = torch.randn(1, 256, device="cuda").bfloat16()
    y, _, _, plan = s.step(_i32([90, 0, 0, 0]), _i32([1] * 4), one.expand(4, 256).contiguous(), 1,
                           fork=(_i32([0, 0, 0]), _i32([1, 2, 3]), _i32([90] * 3)), groups=_i32([0, 4]))
    assert plan.lens.tolist() == [91] * 4
    assert all(torch.equal(y[0], y[i]) for i in range(1, 4))
