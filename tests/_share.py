"""Plain restatement of the calls for shared pages, in loops, for the tests."""


def fork(lens, src, dst, keep, table, refs, page):
    """Python lists and a numpy table, table and refs in place."""
    B, width = table.shape
    old, out, refused = list(lens), list(lens), 0
    made = set()
    for s, d, k in zip(src, dst, keep):
        if not (0 <= s < B and 0 <= d < B) or s == d or old[d] != 0 or old[s] < 0 or d in made:
            refused += 1
            continue
        made.add(d)
        out[d] = min(max(k, 0), old[s], width * page)
        for j in range(-(-out[d] // page)):
            p = int(table[s, j])
            table[d, j] = p
            if 0 <= p < len(refs):
                refs[p] += 1
    return out, [refused]


def own(lens, new, table, stack, count, refs, page):
    """table and refs in place; the new tokens, the copies, [free, refused]."""
    B, width = table.shape
    count = min(max(count, 0), len(stack))
    held = []
    for b in range(B):
        j = lens[b] // page
        p = int(table[b, j]) if new[b] > 0 and lens[b] > 0 and lens[b] % page and j < width else -1
        held.append(p if 0 <= p < len(refs) and refs[p] > 0 else -1)
    writers = {p: [b for b in range(B) if held[b] == p] for p in held if p >= 0}
    keeper = {w[-1] for p, w in writers.items() if len(w) > refs[p]}
    out, copies, used, refused, closed = list(new), [[-1] * 3 for _ in range(B)], 0, 0, False
    for b in range(B):
        if held[b] < 0:
            continue
        if b not in keeper and used >= count:
            closed = True
        if closed:
            out[b] = 0
            refused += 1
        elif b not in keeper:
            to = int(stack[count - 1 - used])
            used += 1
            refs[held[b]] -= 1
            copies[b] = [held[b], to, lens[b] % page]
            table[b, lens[b] // page] = to
    for b in keeper:                             # nobody else holds his page but those refused a copy
        p = held[b]
        refs[p] = sum(out[w] == 0 for w in writers[p] if w != b)
    return out, copies, [count - used, refused]


def release(lens, keep, table, stack, count, refs, page):
    """table, stack (a list) and refs in place."""
    B, width = table.shape
    count = min(max(count, 0), len(stack))
    drops, out = {}, []
    for b in range(B):
        n = lens[b]
        k = min(max(keep[b], 0), n) if n >= 0 else n
        out.append(k)
        for j in range(min(width, -(-max(k, 0) // page)), min(width, -(-max(n, 0) // page))):
            p = int(table[b, j])
            table[b, j] = -1
            if 0 <= p < len(refs):
                drops.setdefault(p, []).append((b, j))
    freed = []
    for p, by in drops.items():
        if len(by) > refs[p]:
            refs[p] = 0
            freed.append((max(by), p))
        else:
            refs[p] -= len(by)
    freed = [p for _, p in sorted(freed)]
    for i, p in enumerate(freed):
        to = count + len(freed) - 1 - i
        if to < len(stack):
            stack[to] = p
    total = count + len(freed)
    return out, [min(total, len(stack)), max(0, total - len(stack))]
