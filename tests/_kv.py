"""Plain 64-bit restatement of the paged-cache operators, on the CPU, for the
tests: loops over requests, pages and heads, no code shared with the library."""
import math

import numpy as np
import torch

E4M3, E5M2, INT8 = 1, 3, 4
EMAX = {E4M3: 8, E5M2: 15, INT8: 6}


def table_of_codes(fmt):
    """The value of each of the 256 codes, from the format's definition."""
    out = np.zeros(256)
    for c in range(256):
        if fmt == INT8:
            out[c] = c - 256 if c >= 128 else c
            continue
        ebits, mbits, bias = (4, 3, 7) if fmt == E4M3 else (5, 2, 15)
        s, e, m = c >> 7, (c >> mbits) & ((1 << ebits) - 1), c & ((1 << mbits) - 1)
        if fmt == E4M3 and (c & 0x7F) == 0x7F:
            v = math.nan
        elif fmt == E5M2 and e == 31:
            v = math.inf if m == 0 else math.nan
        elif e == 0:
            v = m * 2.0 ** (1 - bias - mbits)
        else:
            v = (1 + m / (1 << mbits)) * 2.0 ** (e - bias)
        out[c] = -v if s else v
    return out


TABLES = {f: table_of_codes(f) for f in (E4M3, E5M2, INT8)}


def encode(y, fmt):
    """64-bit values to the nearest code, ties to the even code, saturated; a
    NaN (only a code that no append wrote stands for one) to the code 0x7F."""
    y = np.asarray(y, dtype=np.float64)
    nan = np.isnan(y)
    y = np.where(nan, 0.0, y)
    if fmt == INT8:
        return np.clip(np.rint(y), -128, 127).astype(np.int64).astype(np.uint8)
    t = TABLES[fmt]
    n = 0x7F if fmt == E4M3 else 0x7C            # positive finite codes, ascending
    pos = t[:n]
    a = np.minimum(np.abs(y), pos[-1])
    hi = np.clip(np.searchsorted(pos, a), 1, n - 1)
    lo = hi - 1
    down, up = a - pos[lo], pos[hi] - a
    pick = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(nan, 0x7F, pick | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def scale_code(amax, fmt):
    if not np.isfinite(amax):
        return 255
    if amax == 0:
        return 0
    return int(np.clip(math.frexp(amax)[1] - 1 - EMAX[fmt] + 127, 0, 254))


def append(k, v, ks, vs, fmt, K, V, slots):
    """In place on numpy planes; K, V float64 arrays tokens x heads x d."""
    pages, heads, page, _ = k.shape
    slots = [int(s) for s in slots]
    t = 0
    while t < len(K):
        s = slots[t]
        if s < 0 or s // page >= pages:
            t += 1
            continue
        n = 1
        while t + n < len(K) and slots[t + n] == s + n and (s + n) % page:
            n += 1
        p, off = s // page, s % page
        for codes, scales, x in ((k, ks, K), (v, vs, V)):
            for h in range(heads):
                y = x[t:t + n, h]
                e = scale_code(np.abs(y).max() if np.isfinite(y).all() else np.inf, fmt)
                new = max(e, int(scales[p, h])) if off else e
                if off and new > scales[p, h] and new != 255:
                    old = TABLES[fmt][codes[p, h, :off]]
                    codes[p, h, :off] = encode(old * 2.0 ** (int(scales[p, h]) - new), fmt)
                codes[p, h, off:off + n] = 0 if new == 255 else encode(y * 2.0 ** (127 - new), fmt)
                scales[p, h] = new
        t += n


def values(codes, scale, fmt):
    return TABLES[fmt][codes] * (math.nan if scale == 255 else 2.0 ** (int(scale) - 127))


def attention(Q, k, v, ks, vs, fmt, table, lens, cu, scale, causal=True, window=0):
    """Outputs and, for the error bound, per row: sum_j w_j |v_j| (rows x d),
    the largest error of a score for one unit in 2^-24, the keys visible, and
    the largest |v|.  Q float64 tokens x heads x d; planes numpy."""
    T, Hq, d = Q.shape
    pages, heads, page, _ = k.shape
    G = Hq // heads
    out = np.zeros((T, Hq, d))
    sv = np.zeros((T, Hq, d))
    ex = np.zeros((T, Hq, 1))
    nk = np.zeros((T, Hq, 1))
    vm = np.zeros((T, Hq, 1))
    for b in range(len(lens)):
        a, z, n = int(cu[b]), int(cu[b + 1]), int(lens[b])
        if z == a:
            continue
        for h in range(heads):
            kk, vv = np.zeros((n, d)), np.zeros((n, d))
            for j in range(-(-n // page)):
                p = int(table[b, j])
                m = min(page, n - j * page)
                if p < 0 or p >= pages:
                    kk[j * page:j * page + m] = vv[j * page:j * page + m] = math.nan
                else:
                    kk[j * page:j * page + m] = values(k[p, h, :m], ks[p, h], fmt)
                    vv[j * page:j * page + m] = values(v[p, h, :m], vs[p, h], fmt)
            q = Q[a:z, h * G:(h + 1) * G]
            pos = n - (z - a) + np.arange(z - a)
            j = np.arange(n)
            see = np.ones((z - a, n), bool)
            if causal:
                see &= j <= pos[:, None]
            if window:
                see &= j > pos[:, None] - window
            for i in range(z - a):
                on = see[i]
                if not on.any():
                    continue
                x = scale * (q[i] @ kk[on].T)                # G x keys
                w = np.exp(x - x.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                sl = (a + i, slice(h * G, (h + 1) * G))
                out[sl] = w @ vv[on]
                sv[sl] = w @ np.abs(vv[on])
                ab = np.abs(q[i]) @ np.abs(kk[on]).T
                qm = np.abs(q[i]).max(1)[:, None] * np.abs(kk[on]).sum(1)
                ex[sl] = (abs(scale) * ((d + 4) * ab + 0.5 * qm)).max(1)[:, None] * 2.0 ** -24
                nk[sl] = on.sum()
                vm[sl] = np.abs(vv[on]).max()
    return out, sv, ex, nk, vm


def bound(out, sv, ex, nk, vm, out_dtype):
    """How far an output may be from the exact one.  Each probability is
    rounded to f16 (2^-11 relative; below f16's normal range, 2^-25 of a
    number scaled by 2^7 relative to the largest V scale, whose codes are
    within a factor 2 of the largest value: 2^-31 of that); an error e of the
    scores changes a weight by at most 2 e relative; the exponential and the
    fp32 sums (a chain of a step of 16 keys in every fourth warp, the warps,
    the parts) add 2^-23 each; then the output's own rounding."""
    eps = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[out_dtype]
    rel = 2.0 ** -11 + 2 * ex + (nk / 16 + 64) * 2.0 ** -23
    tiny = {torch.float16: 2.0 ** -25}.get(out_dtype, 0.0)
    return sv * rel + nk * vm * 2.0 ** -31 + np.abs(out) * eps + tiny


def extend(lens, new, table, stack, count, page, max_tokens):
    """Python lists and a numpy table (in place)."""
    B, width = table.shape
    blocks = lambda n: -(-n // page)  # noqa: E731
    lens, out, cu, slots = list(lens), list(lens), [0], []
    count = min(max(count, 0), len(stack))
    free, refused, closed, used = count, 0, False, 0
    for b in range(B):
        n, f = lens[b], new[b]
        if n < 0 or f < 0 or n + f > width * page:
            refused += 1
            cu.append(cu[-1])
            continue
        need = blocks(n + f) - blocks(n)
        if closed or used + need > free or len(slots) + f > max_tokens:
            closed = True
            refused += 1
            cu.append(cu[-1])
            continue
        for j in range(blocks(n), blocks(n + f)):
            table[b, j] = stack[count - 1 - used]
            used += 1
        for pos in range(n, n + f):
            slots.append(int(table[b, pos // page]) * page + pos % page)
        out[b] = n + f
        cu.append(len(slots))
    slots += [-1] * (max_tokens - len(slots))
    return out, cu, slots, [count - used, refused]


def truncate(lens, keep, table, stack, count, page):
    """In place on table and stack (a list)."""
    B, width = table.shape
    count = min(max(count, 0), len(stack))
    freed, out = [], []
    for b in range(B):
        n = lens[b]
        k = min(max(keep[b], 0), n) if n >= 0 else n
        out.append(k)
        for j in range(min(width, -(-max(k, 0) // page)), min(width, -(-max(n, 0) // page))):
            freed.append(int(table[b, j]))
            table[b, j] = -1
    for i, p in enumerate(freed):
        to = count + len(freed) - 1 - i
        if to < len(stack):
            stack[to] = p
    total = count + len(freed)
    return out, [min(total, len(stack)), max(0, total - len(stack))]
