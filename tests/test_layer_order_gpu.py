"""The small kernels come to the GPU while the kernel before them in the stream still
runs, and wait there: what the stream holds before them -- kernels, copies, another
stream's work -- is done and seen when they read, and what comes behind them
sees all of theirs; eagerly and in a graph."""
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
T, HEADS, D = 96, 8, 128
K = HEADS * D


@pytest.fixture(scope="module", autouse=True)
def _built():
    mx.build()


class Chain:
    """x -> rope in place -> norm -> values, on tensors of its own."""

    def __init__(self):
        self.x = torch.empty(T, HEADS, D, dtype=BF16, device="cuda")
        self.positions = torch.empty(T, dtype=torch.int32, device="cuda")
        self.rope = mx.rope_frequencies(D, 10000.0, device="cuda")
        self.weight = torch.empty(K, dtype=torch.float32, device="cuda")
        flat = self.x.view(T, K)
        self.out, _ = mx.mx_rmsnorm_quantize(flat.zero_(), self.weight.zero_(), mx.E4M3)
        self.y = torch.empty(T, K, dtype=BF16, device="cuda")

    def __call__(self):
        mx.mx_rope(self.x, None, self.rope, positions=self.positions, out=(self.x, None))
        mx.mx_rmsnorm_quantize(self.x.view(T, K), self.weight, mx.E4M3, out=self.out)
        mx.mx_dequantize(self.out, BF16, out=self.y)


def _inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, HEADS, D, generator=g, device="cuda").to(BF16),
            torch.randint(0, 4096, (T,), generator=g, device="cuda", dtype=torch.int32),
            torch.randn(K, generator=g, device="cuda"))


def _slow(a):
    """About a millisecond in front of what is written next."""
    for _ in range(4):
        torch.mm(a, a)


def _poison(c):
    c.x.fill_(7.0)
    c.positions.fill_(1)
    c.weight.fill_(-3.0)
    c.y.fill_(5.0)


def _fill(c, src):
    c.x.copy_(src[0])
    c.positions.copy_(src[1])
    c.weight.copy_(src[2])


def _want(c, src):
    torch.cuda.synchronize()
    _fill(c, src)
    torch.cuda.synchronize()
    for step in (lambda: mx.mx_rope(c.x, None, c.rope, positions=c.positions, out=(c.x, None)),
                 lambda: mx.mx_rmsnorm_quantize(c.x.view(T, K), c.weight, mx.E4M3, out=c.out),
                 lambda: mx.mx_dequantize(c.out, BF16, out=c.y)):
        step()
        torch.cuda.synchronize()
    return c.y.clone()


def _same_stream(c, src, heavy):
    _slow(heavy)
    _fill(c, src)


def _side_stream(c, src, heavy):
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    side.wait_stream(main)
    with torch.cuda.stream(side):
        _slow(heavy)
        _fill(c, src)
    c.y.add_(1.0)                                # a kernel of the main stream's, done long before
    main.wait_stream(side)


def _kernels(c, src, heavy):
    _slow(heavy)
    torch.add(src[0], 0.0, out=c.x)
    torch.add(src[1], 0, out=c.positions)
    torch.mul(src[2], 1.0, out=c.weight)


@pytest.mark.parametrize("before", [_same_stream, _side_stream, _kernels])
@pytest.mark.parametrize("captured", [False, True])
def test_what_came_before_is_seen(before, captured):
    c, heavy = Chain(), torch.randn(4096, 4096, device="cuda").to(BF16)
    src = _inputs(0)
    copy = torch.empty_like(c.y)

    def run():
        before(c, src, heavy)
        c()
        copy.copy_(c.y)                          # behind them: sees all of it

    run()                                        # (libraries' first use is outside the capture)
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for seed in range(1, 6):
        for to, new in zip(src, _inputs(seed)):
            to.copy_(new)
        want = _want(c, src)
        _poison(c)
        copy.fill_(9.0)
        graph.replay() if captured else run()
        torch.cuda.synchronize()
        assert torch.equal(copy, want)


def test_two_chains_on_two_streams():
    chains, srcs = [Chain(), Chain()], [_inputs(10), _inputs(11)]
    want = [_want(c, s) for c, s in zip(chains, srcs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    copies = [torch.empty_like(w) for w in want]
    for c in chains:
        _poison(c)
    torch.cuda.synchronize()
    for _ in range(30):
        for c, s, st, y in zip(chains, srcs, streams, copies):
            with torch.cuda.stream(st):
                _fill(c, s)
                c()
                y.copy_(c.y)
    torch.cuda.synchronize()
    for y, w in zip(copies, want):
        assert torch.equal(y, w)
