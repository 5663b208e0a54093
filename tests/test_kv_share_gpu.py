"""mx_kv_fork, mx_kv_own and mx_kv_release against the restatement in loops;
every value is a whole number or a byte that is moved: they are equal."""
import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _share

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    mx.build()
    mx.lib()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Pool:
    """A cache's bookkeeping twice: on the GPU, and in lists."""

    def __init__(self, requests, width, pages, page, heads=2, d=64, fmt=mx.E4M3, seed=0):
        self.rng = np.random.default_rng(seed)
        self.page, self.pages, self.width, self.B = page, pages, width, requests
        self.table = np.full((requests, width), -1, np.int32)
        self.stack = list(self.rng.permutation(pages))
        self.count, self.refs, self.lens = pages, [0] * pages, [0] * requests
        self.cache = mx.empty_kv_cache(fmt, pages, heads, page, d)
        for t in (self.cache.k, self.cache.v, self.cache.k_scales, self.cache.v_scales):
            t.copy_(torch.from_numpy(self.rng.integers(0, 256, tuple(t.shape)).astype(np.uint8)))
        self.planes = [t.cpu().numpy().copy() for t in (self.cache.k, self.cache.v, self.cache.k_scales, self.cache.v_scales)]
        self.g = dict(table=_i32(self.table), stack=_i32(self.stack), count=_i32([self.count, 0]), refs=_i32(self.refs),
                      lens=_i32(self.lens))

    def extend(self, new):
        from tests import _kv
        T = sum(new) + 3
        out, cu, slots, counts = _kv.extend(self.lens, new, self.table, self.stack, self.count, self.page, T)
        plan = mx.mx_kv_extend(self.g["lens"], _i32(new), self.g["table"], self.g["stack"], self.g["count"], self.page, T)
        assert plan.slots.tolist() == slots
        self.lens, self.count = out, counts[0]
        self.g["lens"], self.g["count"] = plan.lens, plan.counts
        self.same()

    def fork(self, src, dst, keep, in_place=False):
        want = _share.fork(self.lens, src, dst, keep, self.table, self.refs, self.page)
        out = mx.KVCut(self.g["lens"], _i32([0])) if in_place else None
        cut = mx.mx_kv_fork(self.g["lens"], _i32(src), _i32(dst), _i32(keep), self.g["table"], self.g["refs"], self.page, out=out)
        self.lens, self.g["lens"] = want[0], cut.lens
        assert cut.counts.tolist() == want[1]
        self.same()

    def own(self, new, in_place=False):
        want = _share.own(self.lens, new, self.table, self.stack, self.count, self.refs, self.page)
        for p, q, n in want[1]:
            if p >= 0:
                for t in self.planes[:2]:
                    t[q, :, :n] = t[p, :, :n]
                for t in self.planes[2:]:
                    t[q] = t[p]
        n = _i32(new)
        out = mx.KVOwn(n, torch.empty(self.B, 3, dtype=torch.int32, device="cuda"), self.g["count"]) if in_place else None
        got = mx.mx_kv_own(self.cache, self.g["lens"], n, self.g["table"], self.g["stack"], self.g["count"], self.g["refs"], out=out)
        assert got.new_tokens.tolist() == want[0] and got.copies.tolist() == want[1] and got.counts.tolist() == want[2]
        self.count, self.g["count"] = want[2][0], got.counts
        for t, w in zip((self.cache.k, self.cache.v, self.cache.k_scales, self.cache.v_scales), self.planes):
            assert (t.cpu().numpy() == w).all()
        self.same()
        return want[0]

    def release(self, keep, in_place=False):
        want = _share.release(self.lens, keep, self.table, self.stack, self.count, self.refs, self.page)
        out = mx.KVCut(self.g["lens"], self.g["count"]) if in_place else None
        cut = mx.mx_kv_release(self.g["lens"], _i32(keep), self.g["table"], self.g["stack"], self.g["count"], self.g["refs"],
                               self.page, out=out)
        assert cut.counts.tolist() == want[1]
        self.lens, self.count = want[0], want[1][0]
        self.g["lens"], self.g["count"] = cut.lens, cut.counts
        self.same()

    def same(self):
        assert self.g["lens"].tolist() == self.lens and (self.g["table"].cpu().numpy() == self.table).all()
        assert self.g["refs"].tolist() == self.refs
        assert self.g["stack"].tolist() == [int(p) for p in self.stack]

    def sound(self):
        """Every page is free, or held by one request more than refs says."""
        held = np.zeros(self.pages, int)
        for b, n in enumerate(self.lens):
            for p in self.table[b, :-(-n // self.page)]:
                held[p] += 1
        free = [int(p) for p in self.stack[:self.count]]
        assert len(set(free)) == len(free) and (held[free] == 0).all() and len(free) + (held > 0).sum() == self.pages
        assert [max(0, h - 1) for h in held] == self.refs


@pytest.mark.parametrize("B,width,page", [(3, 5, 16), (40, 9, 32), (64, 3, 128), (65, 40, 64), (700, 12, 16), (20, 200, 16),
                                          (300, 90, 16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_life_of_shared_pages(B, width, page, in_place):
    p = Pool(B, width, B * width // 2 + 9, page, seed=B)
    rng = p.rng
    p.extend([int(rng.integers(0, width * page // 2)) if b % 4 == 0 else 0 for b in range(B)])
    for step in range(5):
        full = [b for b in range(B) if p.lens[b] > 0]
        free = [b for b in range(B) if p.lens[b] == 0]
        if full and free:
            n = len(free)
            src = [int(x) for x in rng.choice(full, n)]
            dst = [int(x) for x in rng.choice(free, n)]   # the same one now and then: the first is served
            keep = [int(rng.choice([p.lens[s], p.lens[s], rng.integers(-3, p.lens[s] + 9)])) for s in src]
            p.fork(src, dst, keep, in_place)
        p.sound()
        new = [int(x) for x in rng.choice([0, 0, 1, 3], B)]
        new = p.own(new, in_place)
        p.sound()
        p.extend([min(x, width * page - n) for x, n in zip(new, p.lens)])
        p.sound()
        drop = rng.choice([0, 1, 20, 10 ** 6], B, p=[0.5, 0.2, 0.1, 0.2])
        p.release([int(n - x) for n, x in zip(p.lens, drop)], in_place)
        p.sound()
    p.release([0] * B, in_place)
    assert p.count == p.pages and p.refs == [0] * p.pages
    assert mx.mx_last_error() == 0


def test_all_holders_write_and_the_last_keeps():
    p = Pool(5, 2, 20, 16)
    p.extend([20, 0, 0, 0, 0])
    p.fork([0, 0, 0], [1, 2, 4], [20, 18, 5])
    # page two is held by requests 0, 1 and 2, page one by all four
    assert p.own([1, 1, 1, 0, 1]) == [1, 1, 1, 0, 1]
    p.sound()
    assert p.table[4, 0] != p.table[0, 0] and len({p.table[b, 1] for b in range(3)}) == 3


@pytest.mark.parametrize("free", [0, 1, 2, 3])
def test_own_where_pages_run_out(free):
    p = Pool(5, 2, 2 + free, 16)
    p.extend([20, 0, 0, 0, 0])
    p.fork([0] * 4, [1, 2, 3, 4], [20] * 4)
    out = p.own([1] * 5)
    # four copies would be needed; the last holder keeps the page only if all others left it
    assert out == [1] * free + [0] * (5 - free)
    p.sound()


def test_refused_forks():
    p = Pool(6, 3, 12, 16)
    p.extend([40, 7, 0, 0, 0, 0])
    p.fork([0, 0, 0, 9, -1, 2, 0, 3, 1], [2, 2, 1, 3, 3, 4, 6, 3, -5], [40, 30, 7, 1, 1, 1, 1, 1, 1])
    assert p.lens == [40, 7, 40, 0, 0, 0]        # forks 0 and 5 (of an empty request) are served
    p.sound()
    p.fork([], [], [])


def test_holes_and_pages_outside():
    """Entries given back in front of a window are copied as -1; ids outside the cache are
    dropped by release."""
    p = Pool(3, 4, 9, 16)
    p.extend([64, 0, 0])
    p.table[0, 0] = -1
    p.g["table"][0, 0] = -1
    p.fork([0], [2], [60])
    p.table[0, 1] = 999
    p.g["table"][0, 1] = 999
    p.release([0, 0, 0])
    assert (p.g["table"] == -1).all()


def test_release_where_the_stack_has_no_room():
    table, refs = _i32([[3, 4, 5], [3, 6, 7], [4, -1, -1]]), _i32([0, 0, 0, 1, 1, 0, 0, 0])
    stack = _i32([0, 1, -9, -9])
    cut = mx.mx_kv_release(_i32([48, 48, 16]), _i32([0, 0, 0]), table, stack, _i32([2]), refs, 16)
    # freed in the order of those who let go last: 5 (request 0), 3 6 7 (1), 4 (2): the i-th to stack[6 - i]
    assert cut.counts.tolist() == [4, 3] and stack.tolist() == [0, 1, 4, 7] and (table == -1).all() and (refs == 0).all()


@pytest.mark.parametrize("heads,d,page,fmt", [(1, 64, 16, mx.INT8), (8, 128, 128, mx.E4M3), (5, 128, 64, mx.E5M2), (300, 64, 16, mx.E4M3)])
def test_copies_of_whole_heads(heads, d, page, fmt):
    p = Pool(4, 2, 9, page, heads, d, fmt)
    p.extend([2 * page - 1, 0, 1, 0])
    p.fork([0, 2], [1, 3], [2 * page - 1, 1])
    p.own([2, 1, 0, 7])
    p.sound()


def test_many_requests():
    """16384 requests, most of them samples of one prompt."""
    B = 16384
    p = Pool(B, 3, B + 40, 16, 1, 64)
    p.extend([40] + [0] * (B - 1))
    p.fork([0] * (B - 1), list(range(1, B)), [40] * (B - 1))
    p.own([1] * B)
    p.release([0] * B)
    assert p.count == p.pages


def test_captured_and_replayed():
    """A step that ends as it began, recorded once and run again and again."""
    p = Pool(9, 4, 40, 16)
    p.extend([37] + [0] * 8)
    g = p.g
    src, dst, keep, new = _i32([0] * 8), _i32(range(1, 9)), _i32([37] * 8), _i32([0] + [1] * 8)
    back = _i32([37] + [0] * 8)

    def step():
        f = mx.mx_kv_fork(g["lens"], src, dst, keep, g["table"], g["refs"], 16)
        o = mx.mx_kv_own(p.cache, f.lens, new, g["table"], g["stack"], g["count"], g["refs"])
        r = mx.mx_kv_release(f.lens, back, g["table"], g["stack"], o.counts, g["refs"], 16)
        return f, o, r

    before = {k: v.clone() for k, v in g.items()}
    f, o, r = step()
    want = [t.tolist() for t in (f.lens, o.new_tokens, o.copies, o.counts, r.lens, r.counts)]
    assert all(torch.equal(before[k], g[k]) for k in ("table", "refs", "lens"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, o, r = step()
    for _ in range(3):
        graph.replay()
        assert [t.tolist() for t in (f.lens, o.new_tokens, o.copies, o.counts, r.lens, r.counts)] == want
        assert all(torch.equal(before[k], g[k]) for k in ("table", "refs", "lens"))


@pytest.mark.parametrize("B,width", [(1, 9), (64, 70), (700, 40), (3000, 90)])
def test_release_without_sharing_is_truncate(B, width):
    rng = np.random.default_rng(B)
    page, pages = 16, B * width + 7
    lens = rng.integers(0, width * page + 1, B)
    keep = np.where(rng.random(B) < 0.1, -5, lens - rng.choice([0, 1, 3, 40, 10 ** 6], B))
    table = np.full((B, width), -1, np.int32)
    ids, at = rng.permutation(pages), 0
    for b, n in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = np.where(rng.random(m) < 0.2, -1, ids[at:at + m])
        at += m
    stack = np.concatenate([ids[at:], np.full(at, -9)])
    got = []
    for refs in (None, torch.zeros(pages, dtype=torch.int32, device="cuda")):
        t, s, count = _i32(table), _i32(stack), _i32([pages - at])
        if refs is None:
            cut = mx.mx_kv_truncate(_i32(lens), _i32(keep), t, s, count, page)
        else:
            cut = mx.mx_kv_release(_i32(lens), _i32(keep), t, s, count, refs, page)
            assert (refs == 0).all()
        got.append((t, s, cut.lens, cut.counts))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_no_requests():
    none, table = _i32([]), torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    p = Pool(1, 1, 3, 16)
    assert mx.mx_kv_release(none, none, table, p.g["stack"], p.g["count"], p.g["refs"], 16).counts.tolist() == [3, 0]
    assert mx.mx_kv_fork(none, none, none, none, table, p.g["refs"], 16).counts.tolist() == [0]
    assert mx.mx_kv_fork(none, _i32([0]), _i32([1]), _i32([1]), table, p.g["refs"], 16).counts.tolist() == [1]
    own = mx.mx_kv_own(p.cache, none, none, table, p.g["stack"], p.g["count"], p.g["refs"])
    assert own.counts.tolist() == [3, 0] and own.copies.shape == (0, 3)


def test_counts_that_say_too_much_or_too_little():
    """A stack count outside the stack is clipped; a page whose holders are more than its count says is freed
    once, by the last of them, and copied for all but him."""
    table, refs = _i32([[2, 3], [2, 3], [2, 4]]), _i32([0, 0, 1, 0, 0])
    stack = _i32([0, 1, -9, -9, -9])
    cut = mx.mx_kv_release(_i32([32, 32, 32]), _i32([0, 0, 0]), table, stack, _i32([2]), refs, 16)
    assert cut.counts.tolist() == [5, 0] and (refs == 0).all()
    # freed: 3 by request 1, 2 then 4 by request 2
    assert stack.tolist() == [0, 1, 4, 2, 3]
    cut = mx.mx_kv_release(_i32([0]), _i32([0]), _i32([[-1, -1]]), stack, _i32([99]), refs, 16)
    assert cut.counts.tolist() == [5, 0]
    p = Pool(3, 2, 6, 16)
    p.extend([20, 0, 0])
    p.fork([0, 0], [1, 2], [20, 20])
    p.refs[int(p.table[0, 1])] = 1
    p.g["refs"][int(p.table[0, 1])] = 1
    p.own([1, 1, 1])


def test_strided_tables_and_a_stream_argument():
    a, b = Pool(6, 5, 40, 16, seed=3), Pool(6, 5, 40, 16, seed=3)
    wide = torch.full((6, 9), 77, dtype=torch.int32, device="cuda")
    wide[:, 2:7] = b.g["table"]
    b.g["table"] = wide[:, 2:7]
    side = torch.cuda.Stream()
    for p, s in ((a, None), (b, side)):
        p.extend([50, 0, 20, 0, 0, 0])
        torch.cuda.synchronize()
        kw = dict(stream=s)
        f = mx.mx_kv_fork(p.g["lens"], _i32([0, 2, 0]), _i32([1, 3, 5]), _i32([50, 20, 33]), p.g["table"], p.g["refs"], 16, **kw)
        o = mx.mx_kv_own(p.cache, f.lens, _i32([1, 1, 1, 1, 0, 1]), p.g["table"], p.g["stack"], p.g["count"], p.g["refs"], **kw)
        r = mx.mx_kv_release(f.lens, _i32([17, 0, 20, 20, 0, 9]), p.g["table"], p.g["stack"], o.counts, p.g["refs"], 16, **kw)
        torch.cuda.synchronize()
        p.got = f.lens, o.new_tokens, o.copies, o.counts, r.lens, r.counts, p.g["table"], p.g["refs"], p.cache.k, p.cache.v, p.cache.k_scales
    assert all(torch.equal(x, y) for x, y in zip(a.got, b.got))
    assert (wide[:, :2] == 77).all() and (wide[:, 7:] == 77).all()
