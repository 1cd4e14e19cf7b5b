"""The page calls' definitions, row by row in plain Python, shared by the page tests."""
import numpy as np

PAGE = 32


def _clamped(L, mp):
    return min(max(int(L), 0), min(PAGE * mp, 2 ** 31 - 1))


def advance(refs, table, lens, n_new, window=0, sinks=0):
    refs, table = [int(v) for v in refs], np.array(table, dtype=np.int64)
    P, (B, mp) = len(refs), table.shape
    new, count = [], dict(taken=0, released=0, short_of=0, bad=0, clamped=0, pairs=0, reserved=0)
    for b in range(B):
        L, n = _clamped(lens[b], mp), int(n_new[b])
        want = 0 if n < 0 else L + n
        new.append(_clamped(want, mp))
        count["clamped"] += int(L != lens[b] or new[b] != want)
        for j in range(mp):
            e = table[b, j]
            if not 0 <= e < P:
                count["bad"] += int(e != -1)
                table[b, j] = -1
            elif n < 0 or (n > 0 and window > 0 and PAGE * j >= sinks and PAGE * j + PAGE <= L + 1 - window):
                refs[e] -= 1
                count["released"] += 1
                table[b, j] = -1
    free = [p for p in range(P) if refs[p] == 0]
    for b in range(B):
        if n_new[b] < 0:
            continue
        for j in range(_clamped(lens[b], mp) // PAGE, -(-new[b] // PAGE)):
            if table[b, j] < 0:
                if free:
                    table[b, j] = free.pop(0)
                    refs[table[b, j]] = 1
                    count["taken"] += 1
                else:
                    count["short_of"] += 1
    return refs, table, new, dict(count, free_pages=sum(r == 0 for r in refs))


def fork(refs, table, lens, parent):
    old, table = [int(v) for v in refs], np.array(table, dtype=np.int64)
    P, (B, mp), B_out = len(old), table.shape, len(parent)
    refs, free = list(old), [p for p in range(P) if old[p] == 0]
    out, new, pairs, seen = np.full((B_out, mp), -1), [], [], set()
    count = dict(taken=0, released=0, short_of=0, bad=0, pairs=0, reserved=0,
                 clamped=sum(_clamped(L, mp) != L for L in lens))
    for e in table.reshape(-1):
        if 0 <= e < P:
            refs[e] -= 1
    for c, p in enumerate(parent):
        if not 0 <= p < B:
            count["bad"] += int(p >= B)
            new.append(0)
            continue
        L = _clamped(lens[p], mp)
        new.append(L)
        for j in range(mp):
            e = table[p, j]
            if not 0 <= e < P:
                count["bad"] += int(e != -1)
                continue
            if L % PAGE and j == L // PAGE and (p in seen or old[e] != 1):
                if not free:
                    count["short_of"] += 1
                    continue
                pairs.append((int(e), free[0]))
                e = free.pop(0)
                count["taken"] += 1
            out[c, j] = e
            refs[e] += 1
        seen.add(p)
    count["pairs"] = len(pairs)
    pairs += [(-1, -1)] * (B_out - len(pairs))
    return refs, out, new, pairs, dict(count, free_pages=sum(r == 0 for r in refs))


def compact(refs, table):
    refs, table = [int(v) for v in refs], np.array(table, dtype=np.int64)
    P = len(refs)
    live = [p for p in range(P) if refs[p] > 0]
    holes = [p for p in range(len(live)) if refs[p] <= 0]
    pairs = list(zip([p for p in live if p >= len(live)], holes))
    to = {p: p for p in live} | dict(pairs)
    out = np.array([[to.get(int(e), -1) if 0 <= e < P else -1 for e in row] for row in table]).reshape(table.shape)
    bad = sum(int(not 0 <= e < P and e != -1) for e in table.reshape(-1))
    new = [0] * P
    for p in live:
        new[to[p]] = refs[p]
    n = len(pairs)
    pairs += [(-1, -1)] * (max(1, P // 2) - n)
    return new, out, pairs, dict(free_pages=P - len(live), taken=0, released=0, short_of=0, bad=bad, clamped=0, pairs=n,
                                 reserved=0)


def random_state(rng, P, B, mp, share=0.3, window=0, sinks=0):
    """refs, table, lens of a consistent state: rows of random lengths over
    shuffled pages, some of whose full leading pages are shared, the rest of
    a window given back, some references that no row holds."""
    ids = list(rng.permutation(P))
    table, lens, refs = np.full((B, mp), -1), [], [0] * P
    for b in range(B):
        L = int(rng.integers(0, PAGE * mp + 1))
        row = 0
        if b and rng.random() < share:
            row = min(int(rng.integers(0, mp + 1)), L // PAGE, lens[b - 1] // PAGE)
            table[b, :row] = table[b - 1, :row]
        for j in range(row, -(-L // PAGE)):
            if not ids:
                L = min(L, PAGE * j)
                break
            table[b, j] = ids.pop()
        lens.append(L)
        for j in range(mp):
            if window and PAGE * j >= sinks and PAGE * j + PAGE <= L - window:
                table[b, j] = -1
            if table[b, j] >= 0:
                refs[table[b, j]] += 1
    for p in ids[:len(ids) // 8]:
        refs[p] = 1
    return np.array(refs), table, np.array(lens, dtype=np.int64)
