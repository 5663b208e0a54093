"""The 8-bit paged key/value cache on the GPU against the 64-bit restatement
of tests/_kv.py: codes, scales, tables and slots exactly, attention within the
bound derived there."""
import math

import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _kv

pytestmark = pytest.mark.gpu
FMTS = [mx.E4M3, mx.E5M2, mx.INT8]
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    mx.build()
    mx.lib()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _np(t):
    return t.cpu().numpy()


# ------------------------------------------------------------------ pages

def _pages_case(rng, B, page, width, max_new, pages):
    lens = [int(rng.integers(0, width * page // 2 + 1)) for _ in range(B)]
    table = np.full((B, width), -1, np.int32)
    ids = list(rng.permutation(pages))
    for b in range(B):
        for j in range(-(-lens[b] // page)):
            table[b, j] = ids.pop()
    stack = [int(x) for x in ids]
    new = [int(rng.integers(0, max_new + 1)) for _ in range(B)]
    return lens, new, table, stack


def _extend(lens, new, table, stack, count, page, cap):
    t, s = _i32(table), _i32(stack)
    p = mx.mx_kv_extend(_i32(lens), _i32(new), t, s, _i32([count]), page, cap)
    torch.cuda.synchronize()
    assert _np(s).tolist() == list(stack)         # extend only reads the stack
    return p, t


@pytest.mark.parametrize("B,page,width,max_new,cap", [
    (1, 16, 4, 3, 8), (1, 128, 1, 60, 64), (7, 16, 20, 40, 300), (64, 64, 16, 4, 512),
    (513, 32, 12, 9, 5000), (700, 16, 40, 300, 120000), (3000, 16, 6, 5, 16000)])
def test_extend(B, page, width, max_new, cap):
    rng = np.random.default_rng(B)
    lens, new, table, stack = _pages_case(rng, B, page, width, max_new, B * width + 5)
    if B > 4:
        new[1] = new[B // 2] = 0
        lens[2], table[2] = 0, -1
    want_table = table.copy()
    out, cu, slots, counts = _kv.extend(lens, new, want_table, stack, len(stack), page, cap)
    p, t = _extend(lens, new, table, stack, len(stack), page, cap)
    assert _np(p.lens).tolist() == out and _np(p.cu).tolist() == cu
    assert _np(p.slots).tolist() == slots and _np(p.counts).tolist() == counts
    assert (_np(t) == want_table).all()


@pytest.mark.parametrize("free,cap", [(0, 400), (3, 400), (9, 400), (10 ** 6, 37), (10 ** 6, 0), (-5, 400)])
def test_extend_short_of_pages_or_slots(free, cap):
    """The first request that finds no room, and all behind it, are refused."""
    rng = np.random.default_rng(5)
    lens, new, table, stack = _pages_case(rng, 40, 16, 8, 20, 400)
    count = min(free, len(stack))
    want_table = table.copy()
    out, cu, slots, counts = _kv.extend(lens, new, want_table, stack, count, 16, cap)
    p, t = _extend(lens, new, table, stack, count, 16, cap)
    assert counts[1] > 0
    assert _np(p.counts).tolist() == counts and _np(p.lens).tolist() == out
    assert _np(p.cu).tolist() == cu and _np(p.slots).tolist() == slots
    assert (_np(t) == want_table).all()


def test_extend_refuses_malformed_requests_alone():
    table = np.full((5, 2), -1, np.int32)
    lens, new = [0, -3, 0, 0, 0], [5, 1, -1, 33, 32]
    stack = [4, 3, 2, 1, 0]
    want_table = table.copy()
    want = _kv.extend(lens, new, want_table, stack, 5, 16, 64)
    p, t = _extend(lens, new, table, stack, 5, 16, 64)
    assert (_np(p.lens).tolist(), _np(p.cu).tolist(), _np(p.slots).tolist(), _np(p.counts).tolist()) == want
    assert want[3] == [2, 3] and (_np(t) == want_table).all()


@pytest.mark.parametrize("B,page", [(1, 16), (33, 64), (700, 16), (2500, 32)])
def test_truncate_and_extend_undo_each_other(B, page):
    rng = np.random.default_rng(B)
    lens, _, table, stack = _pages_case(rng, B, page, 10, 0, B * 10)
    keep = [int(rng.integers(-1, n + 3)) for n in lens]
    keep[0] = 0
    size = B * 10
    full = stack + [-1] * (size - len(stack))
    want_table, want_stack = table.copy(), list(full)
    out, counts = _kv.truncate(lens, keep, want_table, want_stack, len(stack), page)
    t, s = _i32(table), _i32(full)
    c = mx.mx_kv_truncate(_i32(lens), _i32(keep), t, s, _i32([len(stack)]), page)
    assert _np(c.lens).tolist() == out and _np(c.counts).tolist() == counts
    assert (_np(t) == want_table).all() and _np(s).tolist() == want_stack
    new = [n - o for n, o in zip(lens, out)]
    p = mx.mx_kv_extend(c.lens, _i32(new), t, s, c.counts, page, max(1, sum(new)))
    assert (_np(t) == table).all() and _np(p.lens).tolist() == lens
    assert _np(p.counts).tolist() == [len(stack), 0]


def test_truncate_with_a_full_stack():
    table = np.arange(6, dtype=np.int32).reshape(2, 3)
    want_table, want_stack = table.copy(), [9, -1, -1]
    out, counts = _kv.truncate([48, 40], [0, 16], want_table, want_stack, 1, 16)
    t, s = _i32(table), _i32([9, -1, -1])
    c = mx.mx_kv_truncate(_i32([48, 40]), _i32([0, 16]), t, s, _i32([1]), 16)
    assert counts == [3, 3] and _np(c.counts).tolist() == counts and _np(c.lens).tolist() == out
    assert (_np(t) == want_table).all() and _np(s).tolist() == want_stack


def test_pages_in_place_and_strided_table():
    """Outputs over their inputs, a table that is a part of a wider one, and no
    requests at all."""
    rng = np.random.default_rng(1)
    lens, new, table, stack = _pages_case(rng, 50, 16, 8, 20, 400)
    want_table = table.copy()
    out, cu, slots, counts = _kv.extend(lens, new, want_table, stack, len(stack), 16, 900)
    wide = torch.full((50, 30), 77, dtype=torch.int32, device="cuda")
    t = wide[:, 3:11]
    t.copy_(_i32(table))
    dl, dc = _i32(lens), _i32([len(stack), 0])
    plan = mx.KVPlan(dl, torch.empty(51, dtype=torch.int32, device="cuda"),
                     torch.empty(900, dtype=torch.int64, device="cuda"), dc)
    p = mx.mx_kv_extend(dl, _i32(new), t, _i32(stack), dc, 16, 900, out=plan)
    assert p is plan and _np(dl).tolist() == out and _np(dc).tolist() == counts
    assert _np(p.slots).tolist() == slots and (_np(t) == want_table).all()
    assert (wide[:, :3] == 77).all() and (wide[:, 11:] == 77).all()
    cut = mx.mx_kv_truncate(dl, _i32(lens), t, _i32(stack + [0] * 400), dc, 16, out=mx.KVCut(dl, dc))
    assert _np(cut.lens).tolist() == lens and _np(dc).tolist() == [len(stack), 0]
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    p = mx.mx_kv_extend(none, none, none.view(0, 4), _i32(stack), _i32([3]), 16, 4)
    assert _np(p.cu).tolist() == [0] and _np(p.slots).tolist() == [-1] * 4 and _np(p.counts).tolist() == [3, 0]


# ------------------------------------------------------------------ append

def _planes(cache):
    return [_np(x).copy() for x in (cache.k, cache.v, cache.k_scales, cache.v_scales)]


def _random_cache(fmt, pages, heads, page, d, seed=0):
    """A cache full of garbage, as uninitialised memory may be."""
    g = torch.Generator().manual_seed(seed)
    c = mx.empty_kv_cache(fmt, pages, heads, page, d)
    for t in (c.k, c.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    for t in (c.k_scales, c.v_scales):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    return c


def _check_append(c, K, V, slots):
    want = _planes(c)
    k, v, ks, vs = want
    _kv.append(k, v, ks, vs, c.fmt, _np(K.double()), _np(V.double()), slots)
    mx.mx_kv_append(c, K, V, torch.tensor(slots, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    for got, ref, name in zip(_planes(c), want, ("k", "v", "k_scales", "v_scales")):
        assert (got == ref).all(), (name, np.argwhere(got != ref)[:4])


def _tokens(n, heads, d, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, d, generator=g) * size
    x *= torch.exp2(torch.randint(-3, 4, (n, 1, 1), generator=g).float())
    return x.to(dtype).cuda()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_runs(fmt, page, d, dtype):
    """Whole pages, part pages, single tokens, a run that crosses pages, tokens
    without a slot; then more tokens behind them, small and large (a scale that
    grows makes the earlier codes be rounded again)."""
    c = _random_cache(fmt, 12, 3, page, d)
    at = lambda p, o, n: list(range(p * page + o, p * page + o + n))  # noqa: E731
    first = at(0, 0, page) + at(3, 0, 1) + [-1] + at(5, 0, page // 2 + 1) + at(8, 0, 2 * page) + at(2, 0, 5)
    _check_append(c, _tokens(len(first), 3, d, dtype, 1), _tokens(len(first), 3, d, dtype, 2), first)
    for seed, size in ((3, 0.2), (4, 7.0), (5, 300.0)):
        o = {3: 1, 4: 3, 5: 6}[seed]
        more = at(3, o, 2) + at(5, page // 2 + o, 1) + at(2, 4 + o, 3) + [12 * page, -7]
        _check_append(c, _tokens(len(more), 3, d, dtype, seed, size),
                      _tokens(len(more), 3, d, dtype, 10 + seed, size), more)


@pytest.mark.parametrize("T", [1, 2, 31, 300, 5000])
def test_append_many_tokens(T):
    """Segments of every length the launch chooses from, runs that begin and
    end anywhere in them."""
    rng = np.random.default_rng(T)
    page, heads = 16, 2
    c = _random_cache(mx.E4M3, T + 8, heads, page, 64)
    slots, p = [], 0
    while len(slots) < T:
        n = int(min(T - len(slots), rng.integers(1, 40)))
        slots += list(range(p * page, p * page + n))
        p += -(-n // page)
    _check_append(c, _tokens(T, heads, 64, BF, 1), _tokens(T, heads, 64, BF, 2), slots)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_special_values(fmt):
    """Zeros, the type's extremes, subnormals, NaN and infinities."""
    d, page = 64, 16
    c = _random_cache(fmt, 12, 1, page, d)
    K = torch.zeros(10, 1, d)
    V = torch.zeros(10, 1, d)
    K[1, 0, 3], V[1, 0, 5] = 3.3895e38, -3.3895e38
    K[2, 0, 3], V[2, 0, 5] = 1e-40, -9e-39
    K[3, 0, 0] = math.nan
    V[4, 0, 63] = -math.inf
    K[5, 0] = torch.linspace(-500, 500, d)
    V[6, 0] = torch.linspace(-1.99, 1.99, d)
    K[7, 0, :2] = torch.tensor([-0.0, 5e-39])
    slots = [p * page for p in range(10)]
    _check_append(c, K.bfloat16().cuda(), V.bfloat16().cuda(), slots)
    # behind them: a page stays NaN, a page of zeros takes the new scale, a
    # scale of 2^127 stays, and NaN spoils a good page
    K2, V2 = torch.ones(10, 1, d), torch.full((10, 1, d), 0.01)
    K2[5, 0, 9] = math.inf
    _check_append(c, K2.bfloat16().cuda(), V2.bfloat16().cuda(), [s + 1 for s in slots])
    assert c.k_scales[3, 0] == 255 and c.v_scales[4, 0] == 255 and c.k_scales[5, 0] == 255
    # begun anew, the page is good again
    _check_append(c, K2[:1].bfloat16().cuda(), V2[:1].bfloat16().cuda(), [slots[3]])
    assert c.k_scales[3, 0] != 255


def test_append_strided():
    """Keys and values as slices of a wider projection, and heads first."""
    c = _random_cache(mx.INT8, 6, 4, 16, 64)
    x = _tokens(40, 12, 64, HF, 1)
    _check_append(c, x[:, :4], x[:, 5:9], list(range(40)))
    y = _tokens(4, 20, 64, HF, 2).transpose(0, 1)
    _check_append(c, y, x[::2][:, 8:], list(range(40, 60)))


# ------------------------------------------------------------------ attention

class Setup:
    """Requests over a shuffled pool, written token by token group through
    mx_kv_append, with garbage wherever no token stands."""

    def __init__(self, fmt, page, heads, d, lens, news, dtype=BF, group=2, seed=0, spread=0.0, spare=3):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        ids = rng.permutation(pages)
        width = max(1, max(need)) + 2
        self.table = np.full((len(lens), width), -1, np.int32)
        # behind a request's pages stands anything
        self.table[:, -1] = 10 ** 9
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.cache = _random_cache(fmt, pages, heads, page, d, seed)
        if fmt != mx.INT8:
            nan = 0x7F                            # E4M3's NaN, E5M2's
            self.cache.k[:, :, page // 3:] = nan
            self.cache.v[:, :, page // 3:] = nan
        self.lens, self.news, self.page = list(lens), list(news), page
        slots = [int(self.table[b, j // page]) * page + j % page for b, n in enumerate(lens) for j in range(n)]
        if slots:
            T = len(slots)
            K = _tokens(T, heads, d, dtype, seed + 1)
            V = _tokens(T, heads, d, dtype, seed + 2)
            if spread:
                f = torch.exp2(torch.tensor(rng.uniform(-spread, spread, (T, heads, 1))).float()).cuda()
                V = (V.float() * f.repeat_interleave(1, 0)).to(dtype)
            mx.mx_kv_append(self.cache, K, V, torch.tensor(slots, device="cuda"))
        self.cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.q = _tokens(int(self.cu[-1]), heads * group, d, dtype, seed + 3)

    def run(self, causal=True, window=0, ws=True, out_dtype=None, scale=None, q=None, out=None, max_q=None):
        q = self.q if q is None else q
        w = None
        if ws:
            n = mx.kv_attention_workspace_bytes(q.shape[1], self.cache.k.shape[1], q.shape[2],
                                                max(1, max(self.news)))
            w = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda")
        r = mx.mx_kv_attention(q, self.cache, _i32(self.table), _i32(self.lens), _i32(self.cu),
                               max(self.news) if max_q is None else max_q, causal=causal, window=window,
                               out_dtype=out_dtype, workspace=w, scale=scale, out=out)
        torch.cuda.synchronize()
        assert mx.mx_last_error() == 0
        return r

    def exact(self, causal=True, window=0, scale=None, q=None):
        q = self.q if q is None else q
        k, v, ks, vs = _planes(self.cache)
        return _kv.attention(_np(q.double()), k, v, ks, vs, self.cache.fmt, self.table, self.lens, self.cu,
                             scale or q.shape[2] ** -0.5, causal, window)

    def check(self, causal=True, window=0, ws=True, out_dtype=None, scale=None):
        r = self.run(causal, window, ws, out_dtype, scale)
        e = self.exact(causal, window, scale)
        got = _np(r.double())
        tol = _kv.bound(*e, r.dtype)
        bad = ~(np.abs(got - e[0]) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], e[0][bad][:4], tol[bad][:4])
        return r


EDGES = [0, 1, 15, 16, 17, 31, 33, 64, 127, 128, 129, 250, 257, 400]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention_single_tokens(fmt, d, page, dtype):
    s = Setup(fmt, page, 2, d, EDGES, [1] * len(EDGES), dtype=dtype, group=4)
    for ws in (True, False):
        s.check(ws=ws)
    s.check(out_dtype=F32)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 16, 17, 32])
def test_attention_groups(group):
    s = Setup(mx.E4M3, 32, 3, 64, [5, 130, 300], [1, 2, 1], group=group)
    s.check()


@pytest.mark.parametrize("news", [[2] * 4, [5, 1, 0, 9], [1, 40, 7, 3], [70, 129, 128, 1], [300, 2, 0, 257]])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 50), (False, 50), (True, 1000)])
def test_attention_several_tokens(news, causal, window):
    lens = [max(n, 40 * i + 3) for i, n in enumerate(news)]
    s = Setup(mx.INT8, 16, 2, 64, lens, news, dtype=HF, group=3)
    s.check(causal, window)


def test_attention_rows_that_see_nothing():
    """More rows than keys: the first of them stand before all keys and are
    0; a request without keys gives zeros."""
    s = Setup(mx.E4M3, 16, 2, 64, [3, 0, 40, 0], [9, 4, 60, 1])
    r = s.check()
    assert (r[:6] == 0).all() and (r[9:13] == 0).all() and (r[13:33] == 0).all() and (r[-1] == 0).all()
    assert (s.check(causal=False)[9:13] == 0).all()


@pytest.mark.parametrize("n", [1000, 5000, 20000])
def test_attention_long(n):
    """One request over many SMs; its parts joined."""
    s = Setup(mx.E4M3, 64, 1, 128, [n], [1], group=8)
    a = s.check()
    assert torch.equal(a, s.run())               # whatever order the parts end in


@pytest.mark.parametrize("spread", [6.0, 14.0])
def test_attention_pages_of_very_different_size(spread):
    """V's scale differs by up to 2^28 from token to token and so from page
    to page."""
    s = Setup(mx.E4M3, 16, 2, 64, [300, 77], [2, 1], spread=spread, group=2)
    s.check(out_dtype=F32)


def test_attention_growing_scores():
    """Scores that climb page by page, so that the reference point moves
    again and again; and a negative scale."""
    s = Setup(mx.E4M3, 16, 1, 64, [800], [2], group=4)
    order = torch.arange(800, device="cuda").float()
    K = (torch.ones(800, 1, 64, device="cuda") * (order / 40)[:, None, None]).bfloat16()
    slots = torch.tensor([int(s.table[0, j // 16]) * 16 + j % 16 for j in range(800)], device="cuda")
    V = _tokens(800, 1, 64, BF, 9)
    mx.mx_kv_append(s.cache, K, V, slots)
    s.q = torch.ones_like(s.q)
    s.check(out_dtype=F32)
    s.check(scale=-0.5, out_dtype=F32)


def test_attention_extreme_queries():
    """bf16 rows beyond f16's range, rows of zeros."""
    s = Setup(mx.E4M3, 16, 1, 64, [100, 90, 50], [1, 1, 1], group=2)
    s.q[0] *= 1e30
    s.q[1] *= 1e-30
    s.q[2] = 0
    s.check(scale=1e-31)
    r = s.run()
    assert torch.isfinite(r[1:]).all()


def test_attention_nan_stays_with_its_request():
    """A NaN page, a page id outside the cache: NaN for the rows that see
    them, nothing else touched."""
    lens, news = [100, 100, 100, 100, 40], [1, 1, 2, 1, 1]
    s = Setup(mx.E4M3, 16, 2, 64, lens, news)
    clean = s.run()
    s.cache.k_scales[int(s.table[0, 2]), 1] = 255
    s.cache.v_scales[int(s.table[1, 6]), 0] = 255
    s.table[2, 6] = -1                           # positions 96 ..: both rows see it
    s.table[3, 0] = 10 ** 6
    r = s.run()
    h = lambda x: slice(2 * x, 2 * x + 2)  # noqa: E731
    assert r[0, h(1)].isnan().all() and torch.equal(r[0, h(0)], clean[0, h(0)])
    assert r[1, h(0)].isnan().all() and torch.equal(r[1, h(1)], clean[1, h(1)])
    assert r[2:4].isnan().all() and r[4].isnan().all() and torch.equal(r[5], clean[5])
    # behind the window nothing is followed: a page that no row sees may be gone
    t = Setup(mx.E4M3, 16, 2, 64, [300], [1], seed=4)
    want = t.run(window=60)
    t.table[0, :14] = -1
    assert torch.equal(t.run(window=60), want)
    # a token that a row may not see yet may be anything
    u = Setup(mx.E4M3, 16, 2, 64, [64], [17], seed=5)
    want = u.run()
    u.cache.k_scales[int(u.table[0, 3])] = 255
    u.cache.v_scales[int(u.table[0, 3])] = 255
    got = u.run()
    assert torch.equal(got[:1], want[:1]) and got[1:].isnan().all()


def test_attention_masked_lowest_and_infinite_queries():
    s = Setup(mx.E4M3, 16, 1, 64, [50, 50, 50], [1, 1, 1], dtype=HF, group=2)
    clean = s.run()
    s.q[0, 0] = math.inf
    s.q[1, 1, 7] = math.nan
    r = s.run()
    assert r[0, 0].isnan().all() and r[1, 1].isnan().all()
    assert torch.equal(r[0, 1], clean[0, 1]) and torch.equal(r[1, 0], clean[1, 0]) and torch.equal(r[2], clean[2])


@pytest.mark.parametrize("news", [[1, 2], [40, 70]])
@pytest.mark.parametrize("ws", [True, False])
def test_attention_scores_of_minus_infinity(news, ws):
    """A row whose every score is -infinity is 0 / 0 in both kernels; one that
    sees no key is 0, and the rows beside them stay as they were."""
    s = Setup(mx.E4M3, 16, 1, 64, [500, 700], news, dtype=HF, group=2)
    s.cache.k[..., 5] = 0x38            # 1.0 at value 5 of every key
    clean = s.run(window=100, ws=ws)
    s.q[0, 1, 5] = -math.inf
    s.q[-1, 0, 5] = -math.inf
    r = s.run(window=100, ws=ws)
    assert r[0, 1].isnan().all() and r[-1, 0].isnan().all()
    clean[0, 1] = r[0, 1] = 0
    clean[-1, 0] = r[-1, 0] = 0
    assert torch.equal(r, clean)
    s.lens = [n // 2 - 1 for n in news]                   # the first rows see nothing
    s.q[0, :, 5] = -math.inf
    assert (s.run(ws=ws)[0] == 0).all()


def test_attention_strided_and_offsets_beyond_requests():
    """Q and O inside wider tensors; cu that leaves rows to nobody, goes down
    or beyond Q; lengths beyond the table."""
    s = Setup(mx.E4M3, 16, 2, 64, [100, 33], [3, 2], group=2)
    want = s.run()
    wide = torch.zeros(5, 9, 64, dtype=BF, device="cuda")
    wide[:, 2:6] = s.q
    out = torch.full((5, 7, 64), 5.0, dtype=BF, device="cuda")
    s.run(q=wide[:, 2:6], out=out[:, 1:5])
    assert torch.equal(out[:, 1:5], want) and (out[:, 0] == 5).all() and (out[:, 5:] == 5).all()
    heads_first = s.q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(s.run(q=heads_first), want)
    out = torch.full((5, 4, 64), 5.0, dtype=BF, device="cuda")
    s.cu = np.array([0, 3, 10 ** 6], np.int32)
    got = s.run(out=out)
    assert torch.equal(got[:3], want[:3])
    s.cu, out = np.array([2, 1, 3], np.int32), torch.full((5, 4, 64), 5.0, dtype=BF, device="cuda")
    s.run(out=out)
    assert (out[0] == 5).all() and (out[3:] == 5).all()
    s.lens = [10 ** 9, -4]
    s.cu = np.array([0, 3, 5], np.int32)
    assert s.run().shape == want.shape


@pytest.mark.parametrize("news", [[1], [60]])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_workspace_alignment(news, d):
    """A workspace of exactly the stated size, 16-byte aligned and no more."""
    s = Setup(mx.E4M3, 64, 2, d, [5000], news, group=2)
    want = s.run()
    n = mx.kv_attention_workspace_bytes(4, 2, d, news[0])
    guard = torch.full((n + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    got = mx.mx_kv_attention(s.q, s.cache, _i32(s.table), _i32(s.lens), _i32(s.cu), news[0],
                             workspace=guard[16:16 + n])
    torch.cuda.synchronize()
    assert mx.mx_last_error() == 0 and torch.equal(got, want)
    assert (guard[:16] == 0x5A).all() and (guard[16 + n:] == 0x5A).all()


def test_attention_without_rows():
    s = Setup(mx.E4M3, 16, 2, 64, [10, 0], [0, 0], spare=2)
    q = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    assert mx.mx_kv_attention(q, s.cache, _i32(s.table), _i32(s.lens), _i32(s.cu), 1).shape == (0, 4, 64)
    q = torch.ones(3, 4, 64, dtype=BF, device="cuda")
    out = torch.full_like(q, 5.0)
    s.run(q=q, out=out)
    assert (out == 5).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention_chunks(fmt, d, page, dtype):
    """Chunks of prompts behind what is cached, whole and ragged row tiles
    and key blocks, units of one tile and of two."""
    s = Setup(fmt, page, 2, d, [300, 129, 64, 1, 520], [140, 33, 64, 1, 130], dtype=dtype, group=3)
    for ws in (True, False):
        s.check(ws=ws)
    s.check(causal=False, out_dtype=F32)


def test_attention_chunks_alone_and_many():
    """One unit over all SMs; more units than SMs; units that alternate
    between one tile and two in the same CTA."""
    s = Setup(mx.E4M3, 64, 1, 128, [9000], [40], group=1)
    a = s.check()
    assert torch.equal(a, s.run())
    s = Setup(mx.INT8, 16, 2, 64, [90 + i for i in range(90)], [60 + (37 * i) % 90 for i in range(90)], group=2)
    s.check()
    s.check(ws=False)


def test_attention_chunks_of_special_values():
    """Pages of very different size, growing scores, a negative scale, extreme
    queries, a NaN page and one that is not in the cache, in the kernel for
    many rows."""
    s = Setup(mx.E4M3, 16, 2, 64, [300, 177], [90, 60], spread=14.0, group=2)
    s.check(out_dtype=F32)
    s.check(scale=-0.3, out_dtype=F32)
    s.check(scale=-0.3, causal=False, window=70, out_dtype=F32)
    t = Setup(mx.E4M3, 16, 1, 64, [800], [50], group=4)
    order = torch.arange(800, device="cuda").float()
    K = (torch.ones(800, 1, 64, device="cuda") * (order / 40)[:, None, None]).bfloat16()
    slots = torch.tensor([int(t.table[0, j // 16]) * 16 + j % 16 for j in range(800)], device="cuda")
    mx.mx_kv_append(t.cache, K, _tokens(800, 1, 64, BF, 9), slots)
    t.q = torch.ones_like(t.q)
    t.q[7] = 0
    t.check(out_dtype=F32)
    t.q[3] *= 1e30
    t.q[4] *= 1e-30
    t.check(scale=1e-31)
    u = Setup(mx.E4M3, 16, 2, 64, [300, 100, 150], [40, 60, 33], group=2)
    clean = u.run()
    u.cache.v_scales[int(u.table[0, 17]), 1] = 255        # positions 272 ..: rows 12 .. of 40
    u.table[1, 1] = -1
    r = u.run()
    assert torch.equal(r[:12], clean[:12]) and torch.equal(r[:40, :2], clean[:40, :2])
    assert r[12:40, 2:].isnan().all() and r[40:100].isnan().all() and torch.equal(r[100:], clean[100:])
    w = Setup(mx.E5M2, 16, 1, 128, [600], [40], seed=4)
    want = w.run(window=60)
    w.table[0, :30] = -1                                  # nobody sees before position 500
    assert torch.equal(w.run(window=60), want)


def _check_large(q_len, kv, hq, heads, d, page, fmt, dtype, window=0, requests=1):
    """At the sizes of real prompts: the formula in 64 bits on the GPU for all
    rows, the bound of tests/_kv.py, and the same bits in every run (a race
    between roles that small sizes never lose shows here)."""
    c = mx.empty_kv_cache(fmt, requests * -(-kv // page), heads, page, d)
    g = torch.Generator().manual_seed(kv)
    table = torch.randperm(c.k.shape[0], generator=g).to(torch.int32).view(requests, -1).cuda()
    pos = torch.arange(kv, device="cuda")
    slots = torch.cat([t.long()[pos // page] * page + pos % page for t in table])
    n = requests * kv
    mx.mx_kv_append(c, _tokens(n, heads, d, dtype, 1), _tokens(n, heads, d, dtype, 2), slots)
    Q = _tokens(requests * q_len, hq, d, dtype, 3)
    lens, cu = _i32([kv] * requests), _i32([q_len * i for i in range(requests + 1)])
    ws = torch.empty(mx.kv_attention_workspace_bytes(hq, heads, d, q_len), dtype=torch.uint8, device="cuda")
    for w in (ws, None):
        runs = [mx.mx_kv_attention(Q, c, table, lens, cu, q_len, window=window, workspace=w) for _ in range(6)]
        torch.cuda.synchronize()
        assert mx.mx_last_error() == 0
        assert all(torch.equal(r, runs[0]) for r in runs)
        codes = torch.tensor(_kv.TABLES[fmt], device="cuda")
        for b in range(requests):
            at = kv - q_len + torch.arange(q_len, device="cuda")[:, None]
            see = (pos <= at) & ((pos > at - window) if window else True)
            for h in range(heads):
                def plane(x, s):
                    ids = table[b].long()
                    e = torch.exp2(s[ids, h].double() - 127)[:, None, None]
                    return (codes[x[ids, h].long()] * e).view(-1, d)[:kv]
                k, v = plane(c.k, c.k_scales), plane(c.v, c.v_scales)
                G = hq // heads
                q = Q[b * q_len:(b + 1) * q_len, h * G:(h + 1) * G].double().transpose(0, 1)
                x = (q @ k.T * d ** -0.5).masked_fill(~see, -math.inf)
                p = torch.softmax(x, -1)
                out, sv = p @ v, p @ v.abs()
                ab = (q.abs() @ k.abs().T).masked_fill(~see, 0).amax(-1, keepdim=True)
                qm = q.abs().amax(-1, keepdim=True) * k.abs().sum(-1).max()
                ex = d ** -0.5 * ((d + 4) * ab + 0.5 * qm) * 2.0 ** -24
                e = [t.cpu().numpy() for t in (out, sv, ex, see.sum(-1)[None, :, None].double(),
                                               v.abs().max()[None, None, None])]
                got = runs[0][b * q_len:(b + 1) * q_len, h * G:(h + 1) * G].double().transpose(0, 1)
                assert (np.abs(_np(got) - e[0]) <= _kv.bound(*e, dtype)).all()


@pytest.mark.parametrize("case", [
    (2048, 2048, 32, 8, 128, 64, mx.E4M3, BF), (2048, 2500, 16, 16, 64, 16, mx.INT8, HF),
    (1500, 4000, 8, 2, 128, 128, mx.E5M2, BF, 900), (700, 1900, 12, 4, 128, 32, mx.INT8, HF, 0, 5)])
def test_attention_large_chunks(case):
    _check_large(*case)


@pytest.mark.parametrize("case", [
    (1, 20000, 32, 8, 128, 64, mx.E4M3, BF, 0, 3), (4, 9000, 16, 4, 128, 16, mx.INT8, HF, 5000, 9),
    (1, 7000, 8, 8, 64, 32, mx.E5M2, HF, 0, 20)])
def test_attention_large_decode(case):
    _check_large(*case)


def test_attention_many_requests():
    """More requests than a CTA has threads, most with one token."""
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    s = Setup(mx.INT8, 16, 1, 64, lens, [int(x) for x in rng.integers(0, 3, 700)], group=2)
    s.check()
    s.check(ws=False)
    e = s.exact()                                # and by the kernel for many rows
    assert (np.abs(_np(s.run(max_q=100).double()) - e[0]) <= _kv.bound(*e, BF)).all()


def test_attention_max_q_only_picks_the_kernel():
    s = Setup(mx.E4M3, 32, 2, 128, [0, 1, 77, 300, 500], [3, 1, 70, 1, 20], group=4)
    e = s.exact()
    for most in (1, 2, 70, 5000):
        got = _np(s.run(max_q=most).double())
        assert (np.abs(got - e[0]) <= _kv.bound(*e, BF)).all()


def test_attention_far_offsets():
    """A pool of more than 2^32 bytes a plane, the pages at its end."""
    pages, heads, page, d = 600000, 1, 64, 128
    c = mx.empty_kv_cache(mx.E4M3, pages, heads, page, d)
    n = 200
    table = [pages - 1, 3, pages - 2, 300000]
    slots = torch.tensor([table[j // page] * page + j % page for j in range(n)], device="cuda")
    K, V = _tokens(n, 1, d, BF, 1), _tokens(n, 1, d, BF, 2)
    mx.mx_kv_append(c, K, V, slots)
    q = _tokens(1, 4, d, BF, 3)
    r = mx.mx_kv_attention(q, c, _i32([table]), _i32([n]), _i32([0, 1]), 1)
    chunk = _tokens(40, 4, d, BF, 4)             # the kernel for many rows
    rc = mx.mx_kv_attention(chunk, c, _i32([table]), _i32([n]), _i32([0, 40]), 40)
    small = mx.KVCache(*(x[table].contiguous() for x in (c.k, c.v, c.k_scales, c.v_scales)), mx.E4M3)
    k, v, ks, vs = _planes(small)
    e = _kv.attention(_np(q.double()), k, v, ks, vs, mx.E4M3, np.array([[0, 1, 2, 3]]), [n], [0, 1], d ** -0.5)
    assert (np.abs(_np(r.double()) - e[0]) <= _kv.bound(*e, BF)).all()
    e = _kv.attention(_np(chunk.double()), k, v, ks, vs, mx.E4M3, np.array([[0, 1, 2, 3]]), [n], [0, 40], d ** -0.5)
    assert (np.abs(_np(rc.double()) - e[0]) <= _kv.bound(*e, BF)).all()


def test_attention_of_more_requests_than_the_prompt_kernel_plans():
    """Beyond 16384 requests every call goes through the kernel for few rows."""
    B = 16390
    lens, news = [1 + i % 3 for i in range(B)], [1] * B
    lens[-1], news[-1] = 60, 40
    s = Setup(mx.INT8, 16, 1, 64, lens, news, group=1)
    s.check()


def test_extend_the_most_requests():
    rng = np.random.default_rng(3)
    lens, new, table, stack = _pages_case(rng, 16384, 16, 3, 2, 40000)
    want_table = table.copy()
    want = _kv.extend(lens, new, want_table, stack, len(stack), 16, 33000)
    p, t = _extend(lens, new, table, stack, len(stack), 16, 33000)
    assert (_np(p.lens).tolist(), _np(p.cu).tolist(), _np(p.slots).tolist(), _np(p.counts).tolist()) == want
    assert (_np(t) == want_table).all()


def test_a_step_in_a_graph_and_on_another_stream():
    """truncate, extend, append and attend of a decoding step, captured once
    and replayed on new values; and the same calls on a stream of their own."""
    page, heads, d, B = 16, 2, 64, 6
    lens = [0, 5, 16, 31, 100, 200]
    s = Setup(mx.E4M3, page, heads, d, lens, [1] * B, group=2, spare=30)
    used = set(int(x) for b, n in enumerate(lens) for x in s.table[b, :-(-n // page)])
    free = [p for p in range(s.cache.k.shape[0]) if p not in used]
    size = s.cache.k.shape[0]

    def fresh():
        return dict(table=_i32(s.table), stack=_i32(free + [0] * (size - len(free))), count=_i32([len(free)]),
                    lens=_i32(lens), keep=_i32([n - 1 if n else 0 for n in lens]), new=_i32([2] * B),
                    K=_tokens(2 * B, heads, d, BF, 7), V=_tokens(2 * B, heads, d, BF, 8),
                    q=_tokens(2 * B, 2 * heads, d, BF, 9),
                    cache=mx.KVCache(*(x.clone() for x in (s.cache.k, s.cache.v, s.cache.k_scales,
                                                           s.cache.v_scales)), mx.E4M3))

    ws = torch.empty(mx.kv_attention_workspace_bytes(2 * heads, heads, d, 2), dtype=torch.uint8, device="cuda")

    def step(x):
        cut = mx.mx_kv_truncate(x["lens"], x["keep"], x["table"], x["stack"], x["count"], page)
        plan = mx.mx_kv_extend(cut.lens, x["new"], x["table"], x["stack"], cut.counts, page, 2 * B)
        mx.mx_kv_append(x["cache"], x["K"], x["V"], plan.slots)
        return mx.mx_kv_attention(x["q"], x["cache"], x["table"], plan.lens, plan.cu, 2, workspace=ws)

    want = step(fresh())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x = fresh()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(x)
    side.synchronize()
    assert torch.equal(got, want)
    x = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x)
    for _ in range(3):
        for name, v in fresh().items():
            if name != "cache":
                x[name].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    x["q"].mul_(0.5)
    for name in ("table", "stack", "count", "lens"):
        x[name].copy_(fresh()[name])
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(got, want)
