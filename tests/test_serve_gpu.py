"""The example that serves a layer from the paged cache: every step's
attention against the 64-bit restatement over what the cache then holds."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _kv

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve.py")


@pytest.fixture(scope="module")
def serve():
    mx.build()
    spec = importlib.util.spec_from_file_location("serve", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_steps_of_a_server(serve):
    layer = serve.Layer(256, 6, 2, 64)
    s = serve.Server(layer, requests=3, pages=24, page=16, longest=160, most_new=64, fmt=mx.INT8)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = [0, 0, 0]
    for keep, new in (([0, 0, 0], [64, 5, 0]), ([64, 5, 0], [4, 4, 33]), ([66, 5, 33], [4, 4, 4]),
                      ([0, 7, 36], [20, 1, 1])):
        x = torch.randn(sum(new), 256, device="cuda").bfloat16()
        y, q, o, plan = s.step(i32(keep), i32(new), x, max(new))
        lens = [k + n for k, n in zip(keep, new)]
        assert plan.lens.tolist() == lens and plan.counts.tolist()[1] == 0 and torch.isfinite(y).all()
        c = s.cache
        k, v, ks, vs = [t.cpu().numpy() for t in (c.k, c.v, c.k_scales, c.v_scales)]
        e = _kv.attention(q.double().cpu().numpy(), k, v, ks, vs, mx.INT8, s.table.cpu().numpy(), lens,
                          plan.cu.tolist(), 64 ** -0.5)
        err = np.abs(o.double().cpu().numpy() - e[0])
        assert (err <= _kv.bound(*e, torch.bfloat16)).all()
    held = sum(-(-n // 16) for n in lens)
    assert s.counts.tolist()[0] == 24 - held
    assert mx.mx_last_error() == 0


def test_the_example_runs(serve, capsys):
    serve.main()
    assert "step 11" in capsys.readouterr().out
