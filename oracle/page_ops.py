"""Plain statements of drafted tokens over a paged cache and of the pages that
sequences hold, one sequence after the other (NumPy, fp64 where numbers are
computed)."""
import numpy as np


def tree_attn(q, k, v, scale, seen):
    """One sequence: q [n, HQ, d] against k, v [HK, length, d]; row i sees key j
    where seen[i, j]. Returns o, lse and sum_j p_j |v_j|; rows that see no key:
    zeros and -inf. Keys that no row sees may hold anything."""
    n, HQ, d = q.shape
    group = HQ // k.shape[0]
    o, oa = np.zeros((n, HQ, d)), np.zeros((n, HQ, d))
    lse = np.full((n, HQ), -np.inf)
    for i in range(n):
        at = np.flatnonzero(seen[i])
        if len(at) == 0:
            continue
        for h in range(HQ):
            s = scale * (k[h // group, at] @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            z = e.sum()
            o[i, h] = e @ v[h // group, at] / z
            oa[i, h] = e @ np.abs(v[h // group, at]) / z
            lse[i, h] = m + np.log(z)
    return o, lse, oa


def seen_keys(bits, length):
    """What rows with the masks bits [n, n or more] see of `length` keys: all
    before the last n, of these the ones marked."""
    n = bits.shape[0]
    seen = np.zeros((n, length), dtype=bool)
    for j in range(length):
        t = j - (length - n)
        seen[:, j] = True if t < 0 else bits[:, t]
    return seen


def words_of(bits, words):
    """Masks [rows, tokens] as int32 words: bit t % 32 of word t // 32."""
    rows, tokens = bits.shape
    full = np.zeros((rows, 32 * words), dtype=np.uint8)
    full[:, :min(tokens, 32 * words)] = bits[:, :32 * words]
    return np.packbits(full, axis=1, bitorder="little").view("<u4").astype(np.uint32).view(np.int32)


def ancestors(parents):
    """bits[i, t]: t is i or one of its ancestors; parents[i] < i, -1 for none."""
    bits = np.zeros((len(parents), len(parents)), dtype=bool)
    for i, p in enumerate(parents):
        t = i
        while t >= 0:
            bits[i, t] = True
            t = parents[t]
    return bits


def fork(refs, table, lens, source):
    """Every sequence goes on from source[b]; all at once, in place."""
    old, old_lens = table.copy(), lens.copy()
    for b, s in enumerate(source):
        for p in old[b]:
            if p >= 0:
                refs[p] -= 1
        for p in old[s]:
            if p >= 0:
                refs[p] += 1
        table[b] = old[s]
        lens[b] = old_lens[s]


def resize(refs, table, lens, new_lens, page):
    """Pages given back, then given out, in place; returns the copies and whether
    every sequence was served."""
    B = len(lens)
    pages = [-(-int(n) // page) for n in lens], [-(-int(n) // page) for n in new_lens]
    copies = np.full((B, 2), -1, dtype=np.int32)
    for b in range(B):
        for j in range(pages[1][b], pages[0][b]):
            refs[table[b, j]] -= 1
            table[b, j] = -1
    free = [int(p) for p in np.flatnonzero(refs == 0)]
    left = dict()  # holders of a shared page, as they leave it
    at, all_there = 0, True
    asked = 0
    for b in range(B):
        have, need = pages[0][b], pages[1][b]
        grows_in = new_lens[b] > lens[b] and lens[b] % page != 0
        p = int(table[b, have - 1]) if grows_in else -1
        holders = left.get(p, int(refs[p])) if grows_in else 1
        takes_copy = holders > 1
        want = max(0, need - have) + takes_copy
        shared = grows_in and refs[p] > 1
        if takes_copy:
            left[p] = holders - 1
        asked += want
        if (want or shared) and asked > len(free):
            all_there = False
            continue
        if takes_copy:
            copies[b] = p, free[at]
            table[b, have - 1] = free[at]
            at += 1
        for j in range(have, need):
            table[b, j] = free[at]
            at += 1
        lens[b] = new_lens[b]
    for p in free[:at]:
        refs[p] += 1
    for old, _ in copies:
        if old >= 0:
            refs[old] -= 1
    return copies, all_there


def check_held(refs, table, lens, page):
    """The invariant: counts are the entries', entries are the lengths'."""
    count = np.zeros_like(refs)
    for b, n in enumerate(lens):
        held = -(-int(n) // page)
        assert np.all(table[b, :held] >= 0) and np.all(table[b, held:] == -1)
        for p in table[b, :held]:
            count[p] += 1
    assert np.array_equal(count, refs)


def compact(cache, table, length, n, kept):
    """cache [pages, HK, page, d], in place: of the last n, row kept[i] becomes row i."""
    page = cache.shape[2]
    rows = [cache[table[(length - n + k) // page], :, (length - n + k) % page].copy() for k in kept]
    for i, r in enumerate(rows):
        cache[table[(length - n + i) // page], :, (length - n + i) % page] = r
