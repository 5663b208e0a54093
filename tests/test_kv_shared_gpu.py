"""mx_kv_attention_shared against the 64-bit restatement of attention over the
cache, with mx_kv_attention's bound: the states of the two key sets are joined in
fp32, a few roundings of 2^-24 among the 64 that the bound counts."""
import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx
from tests import _kv

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    mx.build()
    mx.set_shared_bytes(0)                       # short prefixes are shared too
    yield
    mx.set_shared_bytes(-1)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Batch:
    """groups: (common tokens, [(own tokens, rows) of each request]) each; common 0 for requests
    that share nothing (they stand in no group if loose)."""

    def __init__(self, groups, hq, heads, d, page, fmt=mx.E4M3, dtype=BF16, seed=0, spread=2.0):
        rng = np.random.default_rng(seed)
        lens, new, rows, ids = [], [], [], 0
        for common, requests in groups:
            lead = list(range(ids, ids + common // page))
            ids += len(lead)
            for own, n in requests:
                total = common + own
                k = -(-total // page) - len(lead)
                rows.append(lead + list(range(ids, ids + k)))
                ids += k
                lens.append(total)
                new.append(n)
        pages = ids + 2
        order = rng.permutation(pages)
        self.width = max(1, max(len(r) for r in rows))
        table = np.full((len(rows), self.width), -1, np.int32)
        for b, r in enumerate(rows):
            table[b, :len(r)] = order[r]
        if fmt == mx.INT8:
            k, v = (rng.integers(-128, 128, (pages, heads, page, d)).astype(np.int8).view(np.uint8) for _ in "kv")
        else:
            top = 0x7E if fmt == mx.E4M3 else 0x7B
            k, v = (rng.integers(top // 3, top + 1, (pages, heads, page, d)).astype(np.uint8) | (rng.integers(0, 2, (pages, heads, page, d)) << 7).astype(np.uint8)
                    for _ in "kv")
        ref = {mx.E4M3: 127 - 8, mx.E5M2: 127 - 15, mx.INT8: 127 - 7}[fmt]
        ks, vs = ((ref + np.rint(rng.normal(0, spread, (pages, heads)))).astype(np.uint8) for _ in "kv")
        # pages that begin a request's own tokens hold the common rest too: the same values
        for (common, requests), b0 in zip(groups, np.cumsum([0] + [len(r) for _, r in groups[:-1]])):
            j, part = common // page, common % page
            if part and len(requests) > 1:
                p0 = table[b0, j]
                for b in range(b0 + 1, b0 + len(requests)):
                    p = table[b, j]
                    for c, s in ((k, ks), (v, vs)):
                        c[p, :, :part], s[p] = c[p0, :, :part], s[p0]
        self.planes = k, v, ks, vs
        self.fmt, self.heads, self.table, self.lens = fmt, heads, table, lens
        self.cu = np.concatenate([[0], np.cumsum(new)])
        self.most = max(new)
        self.cache = mx.KVCache(*[torch.from_numpy(t).cuda() for t in self.planes], fmt)
        self.q = (torch.randn(int(self.cu[-1]), hq, d, generator=torch.Generator().manual_seed(seed)) * 0.7).to(dtype)
        self.edges = np.cumsum([0] + [len(r) for _, r in groups])
        self.common = [c for c, _ in groups]

    def workspace(self, n_groups=None):
        T, hq, d = self.q.shape
        n = mx.kv_attention_shared_workspace_bytes(T, hq, self.heads, d, self.most, len(self.lens), n_groups or len(self.common))
        assert n > 0
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    def run(self, groups=None, shared=None, ws=True, **kw):
        groups = self.edges if groups is None else groups
        shared = self.common if shared is None else shared
        w = self.workspace(max(1, len(shared))) if ws is True else ws
        return mx.mx_kv_attention_shared(self.q.cuda(), self.cache, _i32(self.table), _i32(self.lens), _i32(self.cu), self.most,
                                         _i32(groups), _i32(shared), workspace=w, **kw)

    def check(self, got, causal=True, scale=None):
        d = self.q.shape[2]
        e = _kv.attention(self.q.double().numpy(), *self.planes, self.fmt, self.table, self.lens, self.cu,
                          d ** -0.5 if scale is None else scale, causal=causal)
        bound = _kv.bound(*e, got.dtype)
        err = np.abs(got.double().cpu().numpy() - e[0])
        assert (err <= bound).all(), (err / np.maximum(bound, 1e-300)).max()
        assert mx.mx_last_error() == 0


CASES = [
    # (groups, hq, heads, d, page, fmt, dtype)
    ([(64, [(5, 1), (9, 1)])], 2, 2, 64, 16, mx.E4M3, BF16),
    ([(128, [(1, 1)] * 4)], 8, 2, 128, 64, mx.E4M3, BF16),
    ([(300, [(17, 1), (200, 1), (33, 2), (64, 0), (40, 4)])], 6, 2, 128, 32, mx.E5M2, F16),
    ([(1, [(3, 1), (2, 2)]), (0, [(40, 1)]), (513, [(1, 1), (90, 1), (130, 1)])], 4, 4, 64, 128, mx.INT8, F16),
    # many rows to a prefix, few to a request
    ([(700, [(7 + 13 * i, 1 + i % 3) for i in range(21)])], 8, 2, 128, 64, mx.E4M3, BF16),
    ([(700, [(7 + 13 * i, 1 + i % 3) for i in range(21)])], 8, 2, 64, 16, mx.INT8, F16),
    ([(333, [(20, 1)] * 40), (0, [(50, 1), (60, 3)]), (256, [(9, 2)] * 9)], 4, 1, 128, 16, mx.E5M2, BF16),
    # many rows to a request
    ([(200, [(90, 40), (70, 66), (150, 1)])], 4, 2, 128, 64, mx.E4M3, BF16),
    ([(128, [(300, 150), (131, 131)]), (0, [(97, 97)])], 2, 1, 64, 32, mx.INT8, F16),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("out_dtype", [F32, None])
@pytest.mark.parametrize("causal", [True, False])
def test_against_64_bits(case, out_dtype, causal):
    groups, hq, heads, d, page, fmt, dtype = CASES[case]
    b = Batch(groups, hq, heads, d, page, fmt, dtype, seed=case)
    got = b.run(causal=causal, out_dtype=out_dtype)
    b.check(got, causal)
    for _ in range(3):                           # the same bits from run to run
        assert torch.equal(b.run(causal=causal, out_dtype=out_dtype), got)


@pytest.mark.parametrize("case", [2, 4, 7])
def test_without_a_workspace_and_without_groups(case):
    groups, hq, heads, d, page, fmt, dtype = CASES[case]
    b = Batch(groups, hq, heads, d, page, fmt, dtype, seed=case)
    plain = mx.mx_kv_attention(b.q.cuda(), b.cache, _i32(b.table), _i32(b.lens), _i32(b.cu), b.most)
    assert torch.equal(b.run(ws=None), plain)
    b.check(b.run(ws=torch.empty(64, dtype=torch.uint8, device="cuda")))
    b.check(b.run(groups=[0], shared=[]))
    b.check(b.run(groups=[0], shared=[], ws=None))


@pytest.mark.parametrize("groups,shared", [
    ([0, 5], [10 ** 9]), ([0, 5], [-7]), ([0, 5], [0]), ([1, 4], [300]), ([0, 2, 5], [300, 100]), ([2, 1, 5], [300, 300]),
    ([-9, 2, 99], [200, 300]), ([0, 1, 2, 3, 4, 5], [300] * 5), ([4, 5], [300]), ([0, 0, 5, 5], [1, 299, 3])])
def test_any_offsets_give_the_same_answer(groups, shared):
    """What a call says of prefixes changes no result."""
    c = CASES[2]
    b = Batch([(300, [(17, 1), (200, 1), (33, 2), (64, 0), (40, 4)])], *c[1:], seed=5)
    b.check(b.run(groups=groups, shared=shared))


def test_rows_that_stand_in_front_of_the_prefix():
    """A request whose rows reach back into the common tokens: less is shared."""
    b = Batch([(256, [(4, 60), (30, 1), (2, 2)])], 4, 2, 128, 32, seed=3)
    b.check(b.run())
    b = Batch([(64, [(1, 65), (3, 1)])], 4, 2, 64, 32, seed=3)   # nothing stands in front of all
    b.check(b.run())


def test_common_tokens_that_end_inside_a_page():
    b = Batch([(300, [(17, 1), (9, 1), (100, 2)])], 4, 2, 64, 128, seed=1)
    b.check(b.run())


def test_strides_outputs_and_rows_of_no_request():
    b = Batch(CASES[4][0], 8, 2, 128, 64, seed=9)
    T = b.q.shape[0]
    wide = torch.randn(T + 5, 3, 8, 136, device="cuda").to(BF16)
    q = wide[:T + 5, 1, :, :128]
    q[:T] = b.q.cuda()
    out = torch.full((T + 5, 8, 160), 7.0, dtype=F16, device="cuda")[..., 16:144]
    got = mx.mx_kv_attention_shared(q, b.cache, _i32(b.table), _i32(b.lens), _i32(b.cu), b.most, _i32(b.edges), _i32(b.common),
                                    out=out, workspace=torch.empty(
                                        mx.kv_attention_shared_workspace_bytes(T + 5, 8, 2, 128, b.most, len(b.lens), 1),
                                        dtype=torch.uint8, device="cuda"))
    b.check(got[:T])
    assert (got[T:] == 7).all()


@pytest.mark.parametrize("many", [False, True])
def test_masked_and_weightless_keys(many):
    """Prefixes whose scores are far below a request's own, and far above; scores of -infinity in one
    set or both; a page with a NaN scale in one request's own keys."""
    n = 12 if many else 2
    for big in (1e4, -1e4):
        b = Batch([(128, [(20 + i, 1) for i in range(n)])], 4, 1, 64, 16, seed=7, spread=0.0)
        b.q[:] = 0
        b.q[..., 0] = 1.0
        k, v, ks, vs = [t.copy() for t in b.planes]
        lead = b.table[0, :8]
        k[..., 0] = 0
        k[lead, ..., 0] = 0x7E if big > 0 else 0xFE     # +-448 times the scale below
        ks[:] = 127 + 4
        b.planes = k, v, ks, vs
        b.cache = mx.KVCache(*[torch.from_numpy(t).cuda() for t in b.planes], b.fmt)
        b.check(b.run(out_dtype=F32))
    # -infinity in the prefix alone: it weighs nothing; in both: NaN
    for both in (False, True):
        b = Batch([(64, [(16, 1) for i in range(n)])], 4, 1, 64, 16, seed=8, spread=0.0, dtype=F16)
        b.q[:] = 0
        b.q[..., 0] = -60000.0
        k, v, ks, vs = [t.copy() for t in b.planes]
        k[..., 0] = 0
        ks[:] = 127
        lead = b.table[0, :4]
        where = np.arange(len(ks)) if both else lead
        k[where, ..., 0] = 0x7E
        ks[where] = 250
        b.planes = k, v, ks, vs
        b.cache = mx.KVCache(*[torch.from_numpy(t).cuda() for t in b.planes], b.fmt)
        got = b.run(out_dtype=F32)
        if both:
            assert torch.isnan(got).all()
        else:
            w = mx.mx_kv_attention(b.q.cuda(), b.cache, _i32(b.table[:, 4:]), _i32([16] * n), _i32(b.cu), 1, out_dtype=F32)
            assert torch.isfinite(got).all() and ((got - w).abs() <= 2.0 ** -10 * w.abs().max()).all()
    # a NaN page of one request's own
    b = Batch([(64, [(16, 1) for i in range(n)])], 4, 1, 64, 16, seed=8)
    k, v, ks, vs = [t.copy() for t in b.planes]
    ks[b.table[1, 4]] = 255
    b.cache = mx.KVCache(*[torch.from_numpy(t).cuda() for t in (k, v, ks, vs)], b.fmt)
    got = b.run(out_dtype=F32)
    assert torch.isnan(got[1]).all() and torch.isfinite(got[[i for i in range(n) if i != 1]]).all()
    assert mx.mx_last_error() == 0


def test_a_page_outside_the_cache():
    b = Batch([(128, [(20, 1), (9, 1), (30, 1)])], 4, 2, 64, 16, seed=2)
    right = b.table[0, 2]
    b.table[:, 2] = 10 ** 6                      # in the prefix
    assert torch.isnan(b.run(out_dtype=F32)).all()
    b.table[1:, 2] = right                       # in one row alone: what the rows agree on is shared
    got = b.run(out_dtype=F32)
    assert torch.isnan(got[0]).all() and torch.isfinite(got[1:]).all()
    b.table[0, 2] = right
    b.table[2, 8] = -1
    got = b.run(out_dtype=F32)
    assert torch.isnan(got[2]).all() and torch.isfinite(got[:2]).all()


def test_captured_and_on_another_stream():
    b = Batch(CASES[6][0], 4, 1, 128, 16, mx.E5M2, seed=6)
    args = (b.q.cuda(), b.cache, _i32(b.table), _i32(b.lens), _i32(b.cu), b.most, _i32(b.edges), _i32(b.common))
    ws = b.workspace()
    want = mx.mx_kv_attention_shared(*args, workspace=ws)
    b.check(want)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws.fill_(255)                            # what stands in a workspace does not matter
        mx.mx_kv_attention_shared(*args, out=out, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_kv_attention_shared(*args, out=out, workspace=ws)
        mx.mx_kv_attention_shared(*args, out=out, workspace=ws)
    for fill in (0, 255):
        ws.fill_(fill)
        out.zero_()
        graph.replay()
        graph.replay()
        assert torch.equal(out, want)
    assert mx.mx_last_error() == 0


def test_a_workspace_of_exactly_the_size_at_a_16_byte_boundary():
    b = Batch(CASES[4][0], 8, 2, 128, 64, seed=4)
    n = b.workspace().numel()
    room = torch.full((n + 16 + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    for at in (0, 16):
        room.fill_(0x5A)
        b.check(b.run(ws=room[at:at + n]))
        assert (room[:at] == 0x5A).all() and (room[at + n:] == 0x5A).all()


@pytest.mark.parametrize("requests,q", [(64, 1), (13, 4)])
def test_serving_sizes(requests, q):
    b = Batch([(2048, [(q + (37 * i) % 256, q) for i in range(requests)])], 32, 8, 128, 64, seed=11)
    b.check(b.run())


def test_prefixes_that_are_not_worth_it():
    """By default a short prefix is read by each request for itself: with a table too short for any other
    the call is mx_kv_attention; behind a wide table the bits are those of entries without prefixes."""
    b = Batch(CASES[2][0], *CASES[2][1:], seed=2)
    plain = mx.mx_kv_attention(b.q.cuda(), b.cache, _i32(b.table), _i32(b.lens), _i32(b.cu), b.most,
                               workspace=b.workspace())
    wide = Batch(CASES[2][0], *CASES[2][1:], seed=2)
    wide.table = np.concatenate([b.table, np.full((len(b.lens), 200000 // 32), -1, np.int32)], 1)
    none = wide.run(shared=[0], out_dtype=F32)
    try:
        mx.set_shared_bytes(-1)
        assert torch.equal(b.run(), plain)
        assert torch.equal(wide.run(out_dtype=F32), none)
    finally:
        mx.set_shared_bytes(0)
    got = wide.run(out_dtype=F32)                # shared, and so summed in another order
    assert not torch.equal(got, none)
    wide.check(got)


def test_the_knob_refuses():
    with pytest.raises(mx.MXError):
        mx.set_shared_bytes(-2)


@pytest.mark.parametrize("case,max_q", [(2, 0), (4, 1), (4, 500), (7, 3), (0, 300)])
def test_any_max_q_gives_the_same_answer(case, max_q):
    """max_q picks the kernels; the rows are what cu says."""
    b = Batch(*CASES[case], seed=case)
    T, hq, d = b.q.shape
    n = mx.kv_attention_shared_workspace_bytes(T, hq, b.heads, d, max(1, max_q), len(b.lens), len(b.common))
    b.most = max_q
    b.check(b.run(ws=torch.empty(n, dtype=torch.uint8, device="cuda")))


@pytest.mark.parametrize("groups,each", [(63, 3), (65, 2), (200, 2)])
def test_many_groups(groups, each):
    b = Batch([(32 + 16 * (g % 3), [(1 + (7 * g + i) % 30, 1 + (g + i) % 2) for i in range(each)]) for g in range(groups)],
              2, 1, 64, 16, seed=groups)
    b.check(b.run())


def test_a_table_with_room_for_far_more():
    """The plan's cluster looks the rows over; other rules between the kernels."""
    b = Batch(CASES[4][0], 8, 2, 128, 64, seed=12)
    want = b.run()
    b.table = np.concatenate([b.table, np.full((len(b.lens), 3000), -1, np.int32)], 1)
    b.check(b.run())
    for at in (0, 5, 10):                        # what the rows agree on ends early, in one of them
        t = Batch(CASES[4][0], 8, 2, 128, 64, seed=12)
        other, mine = t.table[13, at], int(np.setdiff1d(np.arange(len(t.planes[0])), t.table)[0])   # a free page
        for p in t.planes:
            p[mine] = p[other]
        t.table[13, at] = mine
        t.table = np.concatenate([t.table, np.full((len(t.lens), 3000), -1, np.int32)], 1)
        t.cache = mx.KVCache(*[torch.from_numpy(p).cuda() for p in t.planes], t.fmt)
        got = t.run()
        t.check(got)
        assert ((got.double() - want.double()).abs() <= 2.0 ** -6 * want.double().abs().amax()).all()


def test_pages_behind_four_gib():
    """The same pages at the end of a cache of 4.3 GB of keys: the same bits, and copies."""
    b = Batch([(320, [(20, 1), (64, 1), (1, 2)])], 16, 8, 128, 64, seed=5)
    want = b.run()
    pages, small = 66000, b.cache
    n = small.k.shape[0]
    big = mx.empty_kv_cache(b.fmt, pages, 8, 64, 128)
    for t, s in ((big.k, small.k), (big.v, small.v), (big.k_scales, small.k_scales), (big.v_scales, small.v_scales)):
        t[pages - n:] = s
    b.cache, b.table = big, np.where(b.table >= 0, b.table + pages - n, -1).astype(np.int32)
    assert torch.equal(b.run(), want)
    # a request that holds another's last page there writes a copy of it, on the first page and the last
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    page = int(b.table[0, 5])
    refs[page] = 2
    table = _i32(np.stack([b.table[0], b.table[0], b.table[0]]))
    free = [0, int(np.setdiff1d(np.arange(pages - n, pages), b.table)[-1])]
    own = mx.mx_kv_own(big, _i32([340] * 3), _i32([1, 1, 0]), table, _i32(free), _i32([2]), refs)
    assert own.copies.tolist() == [[page, free[1], 20], [page, free[0], 20], [-1] * 3] and refs[page] == 0
    for p in free:
        assert torch.equal(big.k[p, :, :20], big.k[page, :, :20]) and torch.equal(big.v[p, :, :20], big.v[page, :, :20])
        assert torch.equal(big.k_scales[p], big.k_scales[page]) and torch.equal(big.v_scales[p], big.v_scales[page])
    assert mx.mx_last_error() == 0


def test_two_streams_at_once():
    """Calls with workspaces of their own leave each other alone."""
    bs = [Batch(*CASES[c], seed=c) for c in (4, 7)]
    want = [b.run() for b in bs]
    args = [((b.q.cuda(), b.cache, _i32(b.table), _i32(b.lens), _i32(b.cu), b.most, _i32(b.edges), _i32(b.common)), b.workspace())
            for b in bs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mx.mx_kv_attention_shared(*args[i][0], workspace=args[i][1]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


@pytest.mark.parametrize("case", [2, 4, 6, 7])
@pytest.mark.parametrize("scale", [-0.11, 0.0, 0.3])
def test_any_scale(case, scale):
    b = Batch(*CASES[case], seed=case + 30)
    b.check(b.run(scale=scale, out_dtype=F32), scale=scale)


@pytest.mark.parametrize("hq,heads,d", [(5, 1, 128), (16, 1, 64), (20, 4, 64), (3, 3, 128)])
def test_groups_of_heads(hq, heads, d):
    b = Batch([(160, [(33, 1), (7, 2), (64, 3)]), (96, [(1, 1)] * 30)], hq, heads, d, 32, seed=hq)
    b.check(b.run())


def test_a_strided_table_and_a_stream_argument():
    b = Batch(*CASES[6], seed=21)
    want = b.run()
    wide = torch.full((len(b.lens), 64), 12345, dtype=torch.int32, device="cuda")
    wide[:, :b.width] = _i32(b.table)
    side = torch.cuda.Stream()
    args = (b.q.cuda(), b.cache, wide[:, :b.width], _i32(b.lens), _i32(b.cu), b.most, _i32(b.edges), _i32(b.common))
    ws, out = b.workspace(), torch.empty_like(want)
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        out.zero_()
        torch.cuda.synchronize()
        mx.mx_kv_attention_shared(*args, out=out, workspace=ws, stream=s)
        side.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("rows,shares", [(150, True), (260, False)])
def test_requests_with_rows_of_their_own_for_whole_units(rows, shares):
    """By default requests of many rows each are left to themselves, however much they have in common."""
    b = Batch([(96000, [(rows + 9 * i, rows) for i in range(15)])], 1, 1, 64, 128, seed=21)
    plain = mx.mx_kv_attention(b.q.cuda(), b.cache, _i32(b.table), _i32(b.lens), _i32(b.cu), b.most,
                               workspace=b.workspace(), out_dtype=F32)
    assert plain.isfinite().all()
    try:
        mx.set_shared_bytes(-1)
        got = b.run(out_dtype=F32)
    finally:
        mx.set_shared_bytes(0)
    assert torch.equal(got, plain) == (not shares)
    # each weight is off by 2^-11 of itself at most in either, the rest by far less: twice their sum
    assert (got - plain).abs().max() <= 2.0 ** -9 * 448 * 2.0 ** (int(b.planes[3].max()) - 127)


@pytest.mark.parametrize("groups", [70, 600])
def test_many_groups_of_many_rows(groups):
    """More groups than a lane of the prompt kernel's pass looks at once, and more than it looks at at all."""
    b = Batch([(20 + g % 40, [(20 + g % 7, 20), (25 + g % 11, 17)]) for g in range(groups)], 1, 1, 64, 16, seed=groups)
    b.check(b.run())


def test_a_q_with_room_for_more():
    """Rows behind the last request's choose no kernel and are not written; by default a prefix is shared
    all the same."""
    b = Batch([(96000, [(1 + 3 * i, 1) for i in range(15)])], 4, 1, 64, 128, seed=23)
    T = b.q.shape[0]
    q = torch.cat([b.q, torch.full((1500, 4, 64), float("nan"), dtype=BF16)]).cuda()
    n = mx.kv_attention_shared_workspace_bytes(T + 1500, 4, 1, 64, 1, 15, 1)
    args = (b.cache, _i32(b.table), _i32(b.lens), _i32(b.cu), 1)

    def run(shared):
        out = torch.full((T + 1500, 4, 64), 7.0, device="cuda")
        mx.mx_kv_attention_shared(q, *args, _i32([0, 15]), _i32([shared]), out=out,
                                  workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
        assert (out[T:] == 7.0).all()
        return out[:T]

    always = run(10 ** 9)
    try:
        mx.set_shared_bytes(-1)
        got, none = run(10 ** 9), run(0)
    finally:
        mx.set_shared_bytes(0)
    assert torch.equal(got, always) and not torch.equal(got, none)
    b.check(got)


@pytest.mark.parametrize("ended", [[0], [2], [4], [0, 2, 4], [0, 1]])
@pytest.mark.parametrize("left", [-1, 10 ** 6])
def test_requests_without_rows_take_no_sharing_away(ended, left):
    """Requests that have ended, whose rows of the table hold no page or whatever stood there: the others' bits are
    those of a call in which the pages are still in place, and not those without sharing."""
    each = [(17, 1), (200, 1), (33, 2), (64, 1), (40, 4), (9, 1)]
    b = Batch([(300, [(n, 0 if i in ended else r) for i, (n, r) in enumerate(each)])], 6, 2, 128, 32, mx.E5M2, F16, seed=31)
    want, none = b.run(out_dtype=F32), b.run(shared=[0], out_dtype=F32)
    assert not torch.equal(want, none)
    for i in ended:
        b.table[i], b.lens[i] = left, 0
    got = b.run(out_dtype=F32)
    b.check(got)
    assert torch.equal(got, want)


def test_a_group_with_one_request_that_has_rows():
    b = Batch([(300, [(17, 0), (200, 3), (33, 0)]), (0, [(90, 1)])], 4, 2, 64, 32, seed=32)
    b.table[[0, 2]] = -1
    b.lens[0] = b.lens[2] = 0
    b.check(b.run())
    b.cu[:] = 0                                  # nobody has
    b.q = b.q[:1]
    out = torch.full((1, 4, 64), 7.0, device="cuda")
    b.run(out=out, out_dtype=F32)
    assert (out == 7.0).all() and mx.mx_last_error() == 0


@pytest.mark.parametrize("n", [5, 6, 40])
def test_empty_groups_take_no_sharing_away(n):
    """Offsets filled up to a fixed number of groups, that of the requests and more: what is to be shared always is."""
    b = Batch(*CASES[2], seed=33)
    groups = [0] + [5] * n
    got = b.run(groups=groups, shared=[300] + [0] * (n - 1), out_dtype=F32)
    b.check(got)
    assert not torch.equal(got, b.run(groups=groups, shared=[0] * n, out_dtype=F32))
    assert not torch.equal(got, b.run(ws=None, out_dtype=F32))


def _by_default(b, groups, shared):
    """Behind a table with room for far more; the bits without sharing."""
    b.table = np.concatenate([b.table, np.full((len(b.lens), 2000), -1, np.int32)], 1)
    try:
        mx.set_shared_bytes(-1)
        got = b.run(groups=groups, shared=shared, out_dtype=F32)
    finally:
        mx.set_shared_bytes(0)
    b.check(got)
    none = b.run(groups=groups, shared=[0] * len(shared), out_dtype=F32)
    assert not torch.equal(b.run(groups=groups, shared=shared, out_dtype=F32), none)
    return got, none


@pytest.mark.parametrize("n", [0, 1, 15, 300])
@pytest.mark.parametrize("common,worth", [(96000, True), (80000, False)])
def test_what_a_prefix_is_worth_beside_empty_groups(n, common, worth):
    """14 requests are spared 128 bytes for each token: 164 MiB of 96000, 137 of 80000, where 150 are asked by default;
    groups of none and of one request change nothing in that."""
    b = Batch([(common, [(1 + 3 * i, 1) for i in range(15)]), (0, [(200, 1)])], 4, 1, 64, 128, seed=34)
    groups, shared = [0, 15] + [16] * n, [10 ** 9] * (1 + n)
    got, none = _by_default(b, groups, shared)
    assert torch.equal(got, b.run(groups=groups, shared=shared, out_dtype=F32) if worth else none)


def test_small_groups_do_not_make_a_prefix_worth_it():
    """One prefix that saves 68 MiB, a pair that shares nothing and six groups of one request: each group is asked for
    its part of the 150 MiB, that of the groups in which anything can be shared."""
    b = Batch([(40000, [(1 + 3 * i, 1) for i in range(15)]), (0, [(40, 1), (9, 1)])] + [(0, [(30, 1)])] * 6, 4, 1, 64, 128, seed=35)
    got, none = _by_default(b, b.edges, [10 ** 9] * 8)
    assert torch.equal(got, none)


@pytest.mark.parametrize("d", [64, 128])
def test_the_workspace_grows_with_each_argument_but_heads(d):
    size = mx.kv_attention_shared_workspace_bytes
    least = dict(tokens=1, q_heads=8, heads=4, d=d, max_q=1, requests=1, groups=1)
    steps = dict(tokens=[1, 2, 4, 15, 16, 17, 31, 300], q_heads=[4, 8, 12, 32, 64, 128, 256], max_q=[1, 3, 8, 9, 16, 17, 40],
                 requests=[1, 2, 100, 16384], groups=[1, 5, 100, 16384])
    for others in (least, dict(least, tokens=40), dict(least, max_q=20), dict(least, q_heads=64, tokens=7, max_q=3)):
        for name, values in steps.items():
            n = [size(**dict(others, **{name: v})) for v in values]
            assert min(n) > 0 and n == sorted(n)
        assert size(**dict(others, d=64)) < size(**dict(others, d=128))
    # fewer cache heads are more rows to each, for which another kernel wants other room
    n = [size(16, 32, h, d, 1, 4, 1) for h in (1, 2, 8, 32)]
    assert n == sorted(n, reverse=True) and n[0] > n[-1]


def test_many_rows_whose_own_keys_weigh():
    """By default, both passes by the prompt kernel side by side: requests of 150 rows whose own keys, and the prefix's
    last ones, take about half of the softmax, some rows of them against 64 bits.  Of a row's keys, the one at its
    own position weighs 2^-9 or more, where the bound allows 2^-11: a mask that is off by one is seen."""
    n, common, rows = 12, 16384, 150
    b = Batch([(common, [(rows + 9 * i, rows) for i in range(n)])], 4, 4, 128, 128, seed=36, spread=0.5)
    k, v, ks, vs = [t.copy() for t in b.planes]
    ks[:] = 127 - 9                              # |k| < 1
    k[..., 0] = 0
    k[b.table[0, common // 128 - 1], :, -5:, 0] = 0x7E
    for i in range(n):
        k[b.table[i, common // 128:-(-b.lens[i] // 128)], ..., 0] = 0x7E      # 448 * 2^-9
    b.q *= 0.25                                  # scores of 0.1 or so
    b.q[..., 0] = 57.0                           # and 57 * 0.875 / sqrt(128) = 4.4 for those keys: 82 times the weight
    b.planes = k, v, ks, vs
    b.cache = mx.KVCache(*[torch.from_numpy(t).cuda() for t in b.planes], b.fmt)
    plain = mx.mx_kv_attention(b.q.cuda(), b.cache, _i32(b.table), _i32(b.lens), _i32(b.cu), b.most,
                               workspace=b.workspace(), out_dtype=F32)
    try:
        mx.set_shared_bytes(-1)
        got = b.run(out_dtype=F32)
    finally:
        mx.set_shared_bytes(0)
    assert not torch.equal(got, plain)           # it was shared
    some = [(r, i) for r in (0, 1, 7, 11) for i in (0, 1, 63, 127, 128, 149)]
    at = [int(b.cu[r]) + i for r, i in some]
    lens = np.array([b.lens[r] - rows + i + 1 for r, i in some])
    table, one = b.table[[r for r, _ in some]], np.arange(len(some) + 1)

    def exact(lens):
        return _kv.attention(b.q[at].double().numpy(), *b.planes, b.fmt, table, lens, one, 128 ** -0.5)

    e = exact(lens)
    bound = _kv.bound(*e, F32)
    for out in (got, plain):
        assert (np.abs(out[at].double().cpu().numpy() - e[0]) <= bound).all()
    for other in (lens - 1, np.full_like(lens, common)):      # without a row's last key, and without all of its own
        assert (np.abs(exact(other)[0] - e[0]) > bound).any(2).all()
    assert mx.mx_last_error() == 0
