"""The operators around the paged cache's attention in a decoder layer, and the
sizes at which they are measured.

Four kinds of case:

  norm    a residual's addition, the root-mean-square norm of the sum and its MX
          codes and scales (the A operand of a next mx_gemm), and those codes'
          values
  rope    rotary positions of new queries and keys, before the keys go to the cache
  fork    one step of parallel sampling: the samples of the last prompts give their
          pages back, new samples share their prompts' pages, and each gets a
          copy of the last one, which it is about to write
  shared  attention over the cache for groups of requests that share a prefix

With ``own`` false, run() computes the plain form: elementary torch operations
in 32 bits (angles in 64, whole numbers in 64), rounded once at the end.  With
``own`` true it calls the library.
"""
import math

import torch

own = False

E4M3, E2M1, E5M2, INT8 = 1, 2, 3, 4        # the library's format codes
FMT = {"e4m3": E4M3, "e2m1": E2M1, "e5m2": E5M2, "int8": INT8}
EMAX = {"e4m3": 8, "e2m1": 2, "e5m2": 15, "int8": 6}
TOP = {"e4m3": 448.0, "e2m1": 6.0, "e5m2": 57344.0}
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "int8": torch.int8}
EPS = 1e-6


def listed():
    norm = dict(op="norm", x="bf16", res="bf16", fmt="e4m3")
    rope = dict(op="rope", hq=32, heads=8, d=128, rot=128, pairs="halves", dtype="bf16", base=10000.0, factor=1.0)
    fork = dict(op="fork", heads=8, d=128, page=64, fmt="e4m3")
    shared = dict(op="shared", hq=32, heads=8, d=128, page=64, fmt="e4m3", dtype="bf16", alone=0)
    return [
        # one decoding step of 64 requests: latency
        dict(norm, name="norm_64x4096", rows=64, cols=4096),
        # a large batch of prompts, the matrix that the GEMM benchmark quantizes
        dict(norm, name="norm_8192x8192", rows=8192, cols=8192),
        # odd rows, a residual stream in 32 bits, 4-bit codes
        dict(norm, name="norm_4097x5120_e2m1", rows=4097, cols=5120, x="bf16", res="f32", fmt="e2m1"),
        # one new token in each of 64 requests
        dict(rope, name="rope_64", requests=64, most_new=1, longest=8192),
        # whole prompts, 8192 tokens
        dict(rope, name="rope_16x512", requests=16, most_new=512, longest=0),
        # ragged chunks at far positions, scaled for a long context, half of each head, neighbours as pairs
        dict(rope, name="rope_far_half", requests=19, most_new=431, longest=900000, hq=16, heads=4, d=64, rot=32,
             pairs="neighbours", dtype="f16", base=500000.0, factor=8.0),
        # one prompt, sixteen samples: latency
        dict(fork, name="fork_1x16", prompts=1, samples=16, longest=1000),
        # 64 prompts of up to 4096 tokens, eight samples each
        dict(fork, name="fork_64x8", prompts=64, samples=8, longest=4096),
        # four requests behind a short system prompt: latency
        dict(shared, name="shared_4_512", groups=1, each=4, prefix=512, longest=128, q=1),
        # a decoding batch behind one long prefix
        dict(shared, name="shared_64_8192", groups=1, each=64, prefix=8192, longest=512, q=1),
        # eight samples of each of 16 prompts, and requests that share nothing; integer codes, small pages and heads
        dict(shared, name="shared_16x8_ragged_int8", groups=16, each=8, prefix=3000, longest=300, q=1, hq=16, heads=16,
             d=64, page=16, fmt="int8", dtype="f16", alone=5),
        # drafts of 128 requests behind a whole document
        dict(shared, name="shared_128_drafts_32768", groups=1, each=128, prefix=32768, longest=1024, q=4, page=32,
             fmt="e5m2"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "fork", "shared", "shared"])
    if op == "norm":
        cols = 32 * _log(rng, 2, 1024)
        return dict(op=op, rows=_log(rng, 1, min(16384, (1 << 25) // cols)), cols=cols, x=rng.choice(["bf16", "f16", "f32"]),
                    res=rng.choice(["none", "bf16", "f16", "f32"]), fmt=rng.choice(["e4m3", "e5m2", "e2m1"]))
    heads, d = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128])
    group = rng.choice([1, 2, 3, 4, 8]) if heads <= 4 else rng.choice([1, 2, 4])
    if op == "rope":
        requests = _log(rng, 1, 256)
        most = _log(rng, 1, max(1, 8192 * 40 * 128 // (requests * heads * (group + 1) * d)))
        return dict(op=op, requests=requests, most_new=min(most, 4096), longest=rng.choice([0, _log(rng, 1, 1 << 20)]),
                    hq=heads * group, heads=heads, d=d, rot=rng.choice([d, d // 2, d // 4]),
                    pairs=rng.choice(["halves", "neighbours"]), dtype=rng.choice(["bf16", "f16"]),
                    base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 1.0, 4.0]))
    page, fmt = rng.choice([16, 32, 64, 128]), rng.choice(["e4m3", "e5m2", "int8"])
    if op == "fork":
        prompts = _log(rng, 1, 64)
        return dict(op=op, heads=heads, d=d, page=page, fmt=fmt, prompts=prompts, samples=_log(rng, 1, 512 // prompts),
                    longest=_log(rng, 1, 4096 * 64 * 1024 // (max(16, prompts) * heads * d)))
    groups = _log(rng, 1, 16)
    each, q = _log(rng, 1, 128 // groups), rng.choice([1, 1, 1, 2, 4])
    prefix = _log(rng, 64, 32768 // groups)
    return dict(op=op, groups=groups, each=each, prefix=prefix, longest=_log(rng, 1, 1024), q=q, hq=heads * group, heads=heads,
                d=d, page=page, fmt=fmt, dtype=rng.choice(["bf16", "f16"]), alone=rng.choice([0, 0, 3]))


# ------------------------------------------------------------------ sizes

def _spread(n, by=0.6180339887498949):
    return [(i * by) % 1.0 for i in range(1, n + 1)]


def _lengths(case):
    """The whole numbers of a case that its work depends on, from the sizes
    alone, so that work() and prepare() agree; the spread is a fixed
    low-discrepancy sequence.
    rope: each request's tokens before and its new ones; fork: the prompts'
    lengths; shared: the prefixes' tokens, and each request's tokens behind its
    prefix (the new ones among them)."""
    if case["op"] == "rope":
        B = case["requests"]
        old = [int(case["longest"] * x) for x in _spread(B)]
        if case["longest"] == 0 or case["most_new"] == 1:
            return old, [case["most_new"]] * B
        return old, [max(1, int(round(case["most_new"] * x))) for x in _spread(B, 0.7548776662466927)]
    if case["op"] == "fork":
        n = [max(1, int(round(case["longest"] * (0.5 + x / 2)))) for x in _spread(case["prompts"])]
        n[0] = case["longest"]
        return n
    page = case["page"]
    prefix = [case["prefix"]] + [max(page, int(case["prefix"] * (0.5 + x / 2))) for x in _spread(case["groups"] - 1)]
    B = case["groups"] * case["each"] + case["alone"]
    own_ = [case["q"] + int(case["longest"] * x) for x in _spread(B, 0.7548776662466927)]
    return [n // page * page for n in prefix], own_


def work(case):
    if case["op"] == "norm":
        T, C = case["rows"], case["cols"]
        res = 0 if case["res"] == "none" else 2 * SIZE[case["res"]]      # read, and the sum written
        codes = T * C // 2 if case["fmt"] == "e2m1" else T * C
        return {"bytes": T * C * (SIZE[case["x"]] + res) + codes + T * C // 32 + 4 * C, "flops": 5 * T * C}
    if case["op"] == "rope":
        old, new = _lengths(case)
        n = sum(new) * (case["hq"] + case["heads"])
        return {"bytes": 4 * n * case["d"] + 8 * len(new) + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    H, d, page = case["heads"], case["d"], case["page"]
    if case["op"] == "fork":
        # the samples' table entries given back and written, the shared pages'
        # counts twice, and the tokens of each prompt's last page copied
        n, S = _lengths(case), case["samples"]
        entries = S * sum(-(-x // page) for x in n)
        copied = S * sum(x % page for x in n)
        return {"bytes": 4 * 2 * entries + 4 * 4 * sum(x // page for x in n) + 4 * copied * H * d, "flops": 0}
    prefix, own_ = _lengths(case)
    T = case["q"] * len(own_)
    keys = sum(prefix) + sum(own_)
    seen = [prefix[b // case["each"]] if b < case["groups"] * case["each"] else 0 for b in range(len(own_))]
    q = case["q"]
    pairs = sum(q * (s + n) - q * (q - 1) // 2 for s, n in zip(seen, own_))
    return {"bytes": 2 * keys * H * d + 2 * (keys // page + len(own_)) * H + 4 * T * case["hq"] * d,
            "flops": 4 * d * case["hq"] * pairs}


# ------------------------------------------------------------------ inputs

def _pow2(code):
    """2^(code - 127) of UE8M0 codes, in 32 bits."""
    bits = code.to(torch.int32) << 23
    return torch.where(code == 0, torch.full_like(bits, 0x00400000), bits).view(torch.float32)


def _scale_code(amax, fmt):
    e = torch.frexp(amax).exponent.to(torch.int32) - 1 - EMAX[fmt] + 127
    return torch.where(amax == 0, torch.zeros_like(e), e.clamp(0, 254))


def _codes(x, code, fmt):
    """Values and the scale codes of their blocks to 8-bit codes: x / 2^(code -
    127), to the nearest, ties to even, saturated."""
    y = x * _pow2(254 - code)
    if fmt == "int8":
        return y.round().clamp(-128, 127).to(torch.int8).view(torch.uint8)
    return y.clamp(-TOP[fmt], TOP[fmt]).to(CODE[fmt]).view(torch.uint8)


def _values(codes, fmt):
    return codes.view(CODE[fmt]).float()


def _pool(case, g, pages, kind):
    """Codes and scales of a pool of full pages: normal values, whose size
    differs from page to page and head to head."""
    H, d, page = case["heads"], case["d"], case["page"]
    codes = torch.empty(pages, H, page, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, H, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (H * page * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, H, page, d, generator=g, device="cuda")
        if kind == "k":                          # a few channels far larger than the rest
            x[..., ::37] *= 6.0
        x *= torch.exp2(torch.randn(n, H, 1, 1, generator=g, device="cuda") * 0.5)
        s = _scale_code(x.abs().amax((2, 3)), case["fmt"])
        codes[p:p + n] = _codes(x, s[:, :, None, None], case["fmt"])
        scales[p:p + n] = s.to(torch.uint8)
    return codes, scales


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "rope": _prepare_rope, "fork": _prepare_fork, "shared": _prepare_shared}[case["op"]](case, g)


def _prepare_norm(case, g):
    T, C = case["rows"], case["cols"]
    x = torch.randn(T, C, generator=g, device="cuda")
    x *= torch.exp2(torch.randn(T, 1, generator=g, device="cuda"))
    s = dict(case=case, x=x.to(DTYPE[case["x"]]), residual=None,
             weight=1.0 + 0.2 * torch.randn(C, generator=g, device="cuda"))
    if case["res"] != "none":
        r = torch.randn(T, C, generator=g, device="cuda") * 4.0
        r[:, ::101] *= 8.0                       # the residual stream's few large channels
        s["residual"] = r.to(DTYPE[case["res"]])
    return s


def _prepare_rope(case, g):
    old, new = _lengths(case)
    swap = torch.randperm(len(old), generator=g, device="cuda")
    old, new = _ints(old)[swap], _ints(new)[swap]
    cu = torch.zeros(len(old) + 1, dtype=torch.int32, device="cuda")
    cu[1:] = new.cumsum(0)
    hq, h = case["hq"], case["heads"]
    # queries, keys and values side by side, as one projection writes them
    qkv = torch.randn(sum(_lengths(case)[1]), hq + 2 * h, case["d"], generator=g, device="cuda").to(DTYPE[case["dtype"]])
    q, k, _ = qkv.split([hq, h, h], 1)
    return dict(case=case, q=q, k=k, lens=old + new, cu=cu)


def _prepare_fork(case, g):
    """Requests in the order prompt, its samples, next prompt, ...  Each sample
    holds its prompt's whole pages, and a page of its own where the prompt's last one is
    partly filled."""
    P, S, page = case["prompts"], case["samples"], case["page"]
    n = torch.tensor(_lengths(case), dtype=torch.int64, device="cuda")[torch.randperm(P, generator=g, device="cuda")]
    blocks, part = (n + page - 1) // page, (n % page != 0).long()
    need, copies = int(blocks.sum()), int(part.sum()) * S
    pages = need + copies + 9
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(int(blocks.max()), device="cuda")
    first = blocks.cumsum(0) - blocks
    table = torch.where(col < blocks[:, None], ids[(first[:, None] + col).clamp(max=need - 1)], -1)
    table = table.repeat_interleave(S + 1, 0).contiguous()
    req = torch.arange(P * (S + 1), device="cuda")
    prompt, sample = req // (S + 1), req % (S + 1)
    copy = (sample > 0) & (part[prompt] > 0)
    nth = copy.long().cumsum(0) - 1
    at = torch.nonzero(copy)[:, 0]
    table[at, blocks[prompt[at]] - 1] = ids[need + nth[at]]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    whole = col < (n // page)[:, None]
    refs[table[:: S + 1][whole].long()] = S
    stack = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    spare = pages - need - copies
    stack[:spare] = ids[need + copies:]
    lens = n[prompt].int()
    zero = torch.zeros_like(lens)
    child = req[sample > 0].int()
    k, ks = _pool(case, g, pages, "k")
    v, vs = _pool(case, g, pages, "v")
    return dict(case=case, k=k, ks=ks, v=v, vs=vs, table=table, refs=refs, stack=stack, count=_ints([spare]), lens=lens,
                keep=torch.where(sample > 0, zero, lens), src=(prompt * (S + 1))[sample > 0].int(), dst=child,
                take=lens[sample > 0].contiguous(), new=(sample > 0).int())


def _prepare_shared(case, g):
    page, each, G = case["page"], case["each"], case["groups"]
    prefix_, own_ = _lengths(case)
    B = len(own_)
    prefix = torch.tensor(prefix_, dtype=torch.int64, device="cuda")
    own_ = torch.tensor(own_, dtype=torch.int64, device="cuda")[torch.randperm(B, generator=g, device="cuda")]
    req = torch.arange(B, device="cuda")
    group = (req // each).clamp(max=G - 1)
    grouped = req < G * each
    have = torch.where(grouped, prefix[group], 0)
    lead, tail = prefix // page, (own_ + page - 1) // page
    pages = int(lead.sum() + tail.sum()) + 3
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(int((have // page + tail).max()), device="cuda")
    mine = col - (have // page)[:, None]
    at = torch.where(mine < 0, (lead.cumsum(0) - lead)[group][:, None] + col, (lead.sum() + tail.cumsum(0) - tail)[:, None] + mine)
    table = torch.where(mine < tail[:, None], ids[at.clamp(max=pages - 1)], -1).contiguous()
    k, ks = _pool(case, g, pages, "k")
    v, vs = _pool(case, g, pages, "v")
    q = torch.randn(B * case["q"], case["hq"], case["d"], generator=g, device="cuda").to(DTYPE[case["dtype"]])
    return dict(case=case, k=k, ks=ks, v=v, vs=vs, table=table, lens=(have + own_).int(), q=q,
                cu=(torch.arange(B + 1, device="cuda") * case["q"]).int(),
                groups=(torch.arange(G + 1, device="cuda") * each).int(), shared=prefix.int())


# ------------------------------------------------------------------ plain forms

def _plain_norm(s):
    case = s["case"]
    T, C, fmt = case["rows"], case["cols"], case["fmt"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"]
    b = y.view(T, C // 32, 32)
    code = _scale_code(b.abs().amax(2, keepdim=True), fmt)
    z = b * _pow2(254 - code)
    z = _nearest_e2m1(z) if fmt == "e2m1" else z.clamp(-TOP[fmt], TOP[fmt]).to(CODE[fmt]).float()
    values = _returned((z * _pow2(code)).view(T, C), fmt)
    return {"values": values} if s["residual"] is None else {"values": values, "sum": h.to(s["residual"].dtype)}


def _returned(values, fmt):
    """The values that codes stand for, in a type that holds them: a 4-bit code times
    a scale near one has two significant bits, an 8-bit one up to four."""
    return values.to(torch.float8_e5m2 if fmt == "e2m1" else torch.bfloat16)


def _nearest_e2m1(z):
    """To 0, 0.5, 1, 1.5, 2, 3, 4 and 6 with a sign: the nearest, ties to the even code."""
    a = z.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, z)


def _angular(case, dtype):
    """Radians a position of each pair, and what cosines and sines are multiplied by.
    Scaled for a context `factor` times as long as 8192: pairs that turn more than 32 times
    in it keep their frequency, those that turn less than once have it divided, in
    between in proportion."""
    i = torch.arange(case["rot"] // 2, dtype=dtype, device="cuda")
    f = torch.exp(-2.0 * i / case["rot"] * math.log(case["base"]))
    if case["factor"] == 1.0:
        return f, 1.0
    keep = ((8192 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * keep + f / case["factor"] * (1.0 - keep), 0.1 * math.log(case["factor"]) + 1.0


def _rotated(x, cos, sin, case):
    """x: tokens x heads x d; cos, sin: tokens x 1 x rot / 2."""
    half, rot = case["rot"] // 2, case["rot"]
    a, b = (x[..., :half], x[..., half:rot]) if case["pairs"] == "halves" else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat([u, w], -1) if case["pairs"] == "halves" else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    case = s["case"]
    T = s["q"].shape[0]
    cu = s["cu"].long()
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = s["lens"][b] - cu[b + 1] + t
    f, by = _angular(case, torch.float64)
    angle = (pos.double()[:, None] * f)[:, None]
    cos, sin = (torch.cos(angle) * by).float(), (torch.sin(angle) * by).float()
    return {n: _rotated(s[n].float(), cos, sin, case).to(s[n].dtype) for n in "qk"}


def _plain_fork(s):
    case = s["case"]
    page = case["page"]
    lens, keep = s["lens"].long(), s["keep"].long()
    table, refs, stack = s["table"], s["refs"], s["stack"]
    pages, B = refs.numel(), lens.numel()
    blocks = lambda n: (n + page - 1) // page  # noqa: E731
    col = torch.arange(table.shape[1], device="cuda")
    # release: a page whose last holder lets it go is freed, at the place of the last of them
    gone = (col >= blocks(keep)[:, None]) & (col < blocks(lens)[:, None])
    ids = table[gone].long()
    drops = torch.bincount(ids, minlength=pages)
    nth = torch.arange(ids.numel(), device="cuda")
    last = torch.full((pages,), -1, device="cuda").scatter_reduce(0, ids, nth, "amax")
    frees = (drops[ids] > refs[ids]) & (last[ids] == nth)
    freed = ids[frees].int()
    count = s["count"].long()
    stack[(count + freed.numel() - 1 - torch.arange(freed.numel(), device="cuda")).long()] = freed
    count = count + freed.numel()
    refs.copy_((refs - drops).clamp(min=0))
    table.masked_fill_(gone, -1)
    lens = torch.minimum(keep, lens)
    # fork: the samples' rows are their prompts'
    src, dst = s["src"].long(), s["dst"].long()
    n = torch.minimum(s["take"].long(), lens[src])
    rows = torch.where(col < blocks(n)[:, None], table[src], table[dst])
    table[dst] = rows
    refs += torch.bincount(rows[(col < blocks(n)[:, None]) & (rows >= 0)].long(), minlength=pages).int()
    lens[dst] = n
    # own: who is about to write a page that others hold too gets a copy; the
    # last of them keeps it where all of them do
    new = s["new"].long()
    req = torch.arange(B, device="cuda")
    held = table[req, (lens // page).clamp(max=table.shape[1] - 1)].long()
    wants = (new > 0) & (lens % page != 0) & (refs[held.clamp(min=0)] > 0) & (held >= 0)
    who = torch.nonzero(wants)[:, 0]
    p = held[who]
    k = torch.bincount(p, minlength=pages)
    last = torch.full((pages,), -1, device="cuda").scatter_reduce(0, p, who, "amax")
    keeps = (k[p] > refs[p]) & (last[p] == who)
    nth = (~keeps).long().cumsum(0) - 1
    needs = int((~keeps).sum())                  # (there are pages enough)
    to = torch.where(keeps, p, stack[(count - 1 - nth).clamp(min=0)].long())
    copies = torch.full((B, 3), -1, dtype=torch.int32, device="cuda")
    who, p, to = who[~keeps], p[~keeps], to[~keeps]
    copies[who] = torch.stack([p, to, lens[who] % page], 1).int()
    refs.copy_((refs - k).clamp(min=0))
    table[who, lens[who] // page] = to.int()
    some = (torch.arange(page, device="cuda") < (lens[who] % page)[:, None])[:, None, :, None]
    out = {"table": table, "refs": refs, "lens": lens.int(), "new": new.int(), "copies": copies,
           "stack": stack, "counts": torch.cat([count - needs, count.new_zeros(1)]).int()}
    for name in "kv":
        codes, scales = s[name], s[name + "s"]
        codes[to] = torch.where(some, codes[p], codes[to])
        scales[to] = scales[p]
        out[name], out[name + "s"] = codes.view(CODE[case["fmt"]]), scales
    return out


def _plain_shared(s):
    case = s["case"]
    H, d, page, q, G = case["heads"], case["d"], case["page"], case["q"], case["hq"] // case["heads"]
    prefix, own_ = _lengths(case)
    B, each = len(own_), case["each"]

    def values(codes, scales, ids):              # ids ... x blocks -> ... x heads x keys x d
        x = _values(codes[ids], case["fmt"]) * _pow2(scales[ids])[..., None, None]
        return x.transpose(-4, -3).flatten(-3, -2)

    out = torch.empty_like(s["q"])
    sets = [(g * each, (g + 1) * each, n) for g, n in enumerate(prefix)] + [(b, b + 1, 0) for b in range(case["groups"] * each, B)]
    for b0, b1, n in sets:
        R, lead = b1 - b0, n // page
        x = s["q"][b0 * q:b1 * q].float().view(R, q, H, G, d).permute(2, 0, 3, 1, 4)      # H R G q d
        ids = s["table"][b0:b1, lead:].clamp(min=0).long()
        mine = s["lens"][b0:b1].long() - n
        j = torch.arange(ids.shape[1] * page, device="cuda")
        see = (j <= (mine - q)[:, None, None] + torch.arange(q, device="cuda")[:, None])[None, :, None]
        k2 = values(s["k"], s["ks"], ids).transpose(0, 1)                                 # H R keys d
        x2 = torch.einsum("hrgid,hrjd->hrgij", x, k2) * d ** -0.5
        x2 = x2.masked_fill(~see, -math.inf)
        top = x2.amax(-1, keepdim=True)
        first = s["table"][b0, :lead].long()
        if n:
            x1 = torch.einsum("hrgid,hjd->hrgij", x, values(s["k"], s["ks"], first)) * d ** -0.5
            top = torch.maximum(top, x1.amax(-1, keepdim=True))
        p2 = torch.exp(x2 - top)
        # pages hold garbage behind a request's last token
        v2 = torch.where((j < mine[:, None])[None, :, :, None], values(s["v"], s["vs"], ids).transpose(0, 1), 0.0)
        o, total = torch.einsum("hrgij,hrjd->hrgid", p2, v2), p2.sum(-1, keepdim=True)
        if n:
            p1 = torch.exp(x1 - top)
            o = o + torch.einsum("hrgij,hjd->hrgid", p1, values(s["v"], s["vs"], first))
            total = total + p1.sum(-1, keepdim=True)
        out[b0 * q:b1 * q] = (o / total).permute(1, 3, 0, 2, 4).reshape(R * q, H * G, d).to(out.dtype)
    return out


# ------------------------------------------------------------------ one pass

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "rope": _plain_rope, "fork": _plain_fork, "shared": _plain_shared}[op](s)
    import block_scaled_quantized_mx_gb300 as mx
    if op == "norm":
        out, h = mx.mx_rmsnorm_quantize(s["x"], s["weight"], FMT[case["fmt"]], residual=s["residual"], eps=EPS)
        values = mx.mx_dequantize(out, out_dtype=torch.bfloat16)
        if case["fmt"] == "e2m1":
            values = _returned(values, "e2m1")
        return {"values": values} if h is None else {"values": values, "sum": h}
    if op == "rope":
        if "rope" not in s:
            s["rope"] = mx.rope_frequencies(case["rot"], case["base"], factor=case["factor"], original=8192)
        q, k = mx.mx_rope(s["q"], s["k"], s["rope"], lens=s["lens"], cu=s["cu"], neighbours=case["pairs"] == "neighbours")
        return {"q": q, "k": k}
    if "cache" not in s:
        s["cache"] = mx.KVCache(s["k"], s["v"], s["ks"], s["vs"], FMT[case["fmt"]])
    if op == "fork":
        cut = mx.mx_kv_release(s["lens"], s["keep"], s["table"], s["stack"], s["count"], s["refs"], case["page"])
        fork = mx.mx_kv_fork(cut.lens, s["src"], s["dst"], s["take"], s["table"], s["refs"], case["page"])
        own_ = mx.mx_kv_own(s["cache"], fork.lens, s["new"], s["table"], s["stack"], cut.counts, s["refs"])
        code = CODE[case["fmt"]]
        return {"table": s["table"], "refs": s["refs"], "lens": fork.lens, "new": own_.new_tokens, "copies": own_.copies,
                "stack": s["stack"], "counts": own_.counts, "k": s["k"].view(code), "ks": s["ks"], "v": s["v"].view(code),
                "vs": s["vs"]}
    if "workspace" not in s:
        n = mx.kv_attention_shared_workspace_bytes(s["q"].shape[0], case["hq"], case["heads"], case["d"], case["q"],
                                                   s["lens"].numel(), case["groups"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return mx.mx_kv_attention_shared(s["q"], s["cache"], s["table"], s["lens"], s["cu"], case["q"], s["groups"], s["shared"],
                                     workspace=s["workspace"])


# ------------------------------------------------------------------ 64 bits

def _exact_norm(s):
    case = s["case"]
    T, C, fmt = case["rows"], case["cols"], case["fmt"]
    low, bits = {"e4m3": (-6, 3), "e5m2": (-14, 2), "e2m1": (0, 1)}[fmt]
    h = s["x"].double() + (0.0 if s["residual"] is None else s["residual"].double())
    y = h / torch.sqrt(h.square().sum(1, keepdim=True) / C + EPS) * s["weight"].double()
    y = y.view(T, -1, 32)
    top = torch.frexp(y.abs().amax(2, keepdim=True)).exponent.double() - 1
    unit = torch.exp2((top - EMAX[fmt]).clamp(-127, 127))
    z = y / unit
    step = torch.exp2((torch.frexp(z.abs()).exponent.double() - 1).clamp(min=low) - bits)
    values = ((torch.round(z / step) * step).clamp(-TOP[fmt], TOP[fmt]) * unit).view(T, C)
    return {"values": values} if s["residual"] is None else {"values": values, "sum": h}


def _exact_rope(s):
    case = s["case"]
    f, by = _angular(case, torch.float64)
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    pos = torch.cat([torch.arange(n - (z - a), n, device="cuda") for a, z, n in zip(cu, cu[1:], lens)]).double()
    turn = torch.polar(torch.full((pos.numel(), 1, f.numel()), by, dtype=torch.float64, device="cuda"),
                       (pos[:, None] * f)[:, None])
    out = {}
    for n in "qk":
        x, rot = s[n].double(), case["rot"]
        split = (2, rot // 2) if case["pairs"] == "halves" else (rot // 2, 2)
        axis = -2 if case["pairs"] == "halves" else -1
        z = x[..., :rot].reshape(*x.shape[:2], *split)
        z = torch.complex(z.select(axis, 0), z.select(axis, 1)) * turn
        out[n] = torch.cat([torch.stack([z.real, z.imag], axis).reshape(*x.shape[:2], rot), x[..., rot:]], -1)
    return out


def _exact_shared(s):
    case = s["case"]
    page, H, d = case["page"], case["heads"], case["d"]
    G = case["hq"] // H
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for b, n in enumerate(lens):
        a, z = cu[b], cu[b + 1]
        ids = s["table"][b, :-(-n // page)].long()
        k, v = ((codes[ids].view(CODE[case["fmt"]]).double() * torch.exp2(scales[ids].double() - 127)[..., None, None])
                .transpose(0, 1).reshape(H, -1, d)[:, :n] for codes, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])))
        q = s["q"][a:z].double().view(z - a, H, G, d)
        x = torch.einsum("ihgd,hjd->hgij", q, k) / math.sqrt(d)
        late = torch.arange(n, device="cuda") > (torch.arange(z - a, device="cuda") + n - (z - a))[:, None]
        out[a:z] = torch.einsum("hgij,hjd->ihgd", torch.softmax(x.masked_fill(late, -math.inf), -1), v).reshape(z - a, H * G, d)
    return out


def exact(case, seed):
    if case["op"] == "fork":
        return None                              # whole numbers, and codes that are moved
    if case["op"] == "shared" and work(case)["flops"] > 4e11:
        return None
    return {"norm": _exact_norm, "rope": _exact_rope, "shared": _exact_shared}[case["op"]](prepare(case, seed))
