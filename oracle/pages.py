"""fp64 numpy reference of the calls on pages that requests share, and of attention of many query
rows over a paged cache. Plain loops, from the definitions."""
import numpy as np

from . import _f64, _i32
from .attention import visible


def _held(n_tokens, block, width):
    return min(-(-max(int(n_tokens), 0) // block), width)


def fork(src, dst, lens, table, block, shares, free):
    """One fork after another. Returns (table, shares, copy_src, copy_dst, counts)."""
    table, shares, free = _i32(table).copy(), _i32(shares).copy(), [int(x) for x in _i32(free)]
    rows, width = table.shape
    copy, asked = [], 0
    for s, t, x in zip(_i32(src), _i32(dst), _i32(lens)):
        pair = (-1, -1)
        if 0 <= s < rows and 0 <= t < rows and s != t:
            x = min(max(int(x), 0), width * block)
            whole = x // block
            for p in range(whole):
                table[t, p] = table[s, p]
                if 0 <= table[s, p] < len(shares):
                    shares[table[s, p]] += 1
            if x % block:
                page, got = int(table[s, whole]), -1
                if 0 <= page < len(shares):
                    got = free[asked] if asked < len(free) else -1
                    asked += 1
                table[t, whole] = got
                if got >= 0:
                    pair = (page, got)
        copy.append(pair)
    return (table, shares, np.array([p[0] for p in copy], dtype=np.int64),
            np.array([p[1] for p in copy], dtype=np.int64),
            np.array([asked, min(asked, len(free))]))


def free(rows, lens, table, block, shares, max_freed):
    """Returns (table, shares, freed, counts)."""
    table, shares = _i32(table).copy(), _i32(shares).copy()
    gone = set()
    for r, x in zip(_i32(rows), _i32(lens)):
        if not 0 <= r < table.shape[0]:
            continue
        for p in range(_held(x, block, table.shape[1])):
            page, table[r, p] = int(table[r, p]), -1
            if not 0 <= page < len(shares):
                continue
            if shares[page] > 0:
                shares[page] -= 1
            else:
                gone.add(page)
    out = sorted(gone)[:max_freed]
    return (table, shares, np.array(out + [-1] * (max_freed - len(out)), dtype=np.int64),
            np.array([len(gone)]))


def compact(lens, table, block, shares, max_copies):
    """Returns (table, shares, copy_src, copy_dst, counts)."""
    table, shares = _i32(table).copy(), _i32(shares).copy()
    n = len(shares)
    at = [(i, p) for i in range(table.shape[0]) for p in range(_held(lens[i], block,
                                                                     table.shape[1]))
          if 0 <= table[i, p] < n]
    live = {int(table[i, p]) for i, p in at}
    src = [x for x in sorted(live) if x >= len(live)]
    dst = [x for x in range(len(live)) if x not in live]
    to = dict(list(zip(src, dst))[:max_copies])
    for i, p in at:
        table[i, p] = to.get(int(table[i, p]), table[i, p])
    for a, b in to.items():
        shares[b], shares[a] = shares[a], 0
    pad = [-1] * (max_copies - len(to))
    return (table, shares, np.array(list(to) + pad, dtype=np.int64),
            np.array(list(to.values()) + pad, dtype=np.int64), np.array([len(live), len(src)]))


def attend_rows(q, k, v, pos, lim, scale):
    """Query rows q [R, d], row i over the keys with pos < lim[i]: (outputs, mean |v| under the
    weights, largest absolute score sum of each row). A row without keys: zeros."""
    keep = np.asarray(pos)[None, :] < np.asarray(lim)[:, None]
    s = np.where(keep, scale * (q @ k.T), -np.inf)
    top = s.max(axis=1, initial=-np.inf, keepdims=True)
    e = np.exp(s - np.where(np.isinf(top), 0.0, top))
    total = e.sum(axis=1, keepdims=True)
    p = e / np.where(total == 0, 1.0, total)
    sums = np.where(keep, abs(scale) * (np.abs(q) @ np.abs(k).T), 0.0)
    return p @ v, p @ np.abs(v), sums.max(axis=1, initial=0.0)


def _keys(cache_k, cache_v, row, n, head, block):
    seen = visible(row, n, block, cache_k.shape[0])
    pos = np.array([x[0] for x in seen], dtype=np.int64)
    page = np.array([x[1] for x in seen], dtype=np.int64)
    off = np.array([x[2] for x in seen], dtype=np.int64)
    return pos, cache_k[page, head, off], cache_v[page, head, off]


def prefill(q, k_cache, v_cache, table, cu, lens, scale):
    """Packed q [T, H, d], causal: a request's new tokens are its last cu[i + 1] - cu[i]. Returns
    (o, mean |v|, absolute score sums [T, H])."""
    q, kc, vc = _f64(q), _f64(k_cache), _f64(v_cache)
    table, lens, cu = _i32(table), _i32(lens), _i32(cu)
    T, H, d = q.shape
    kv, block = kc.shape[1], kc.shape[2]
    G = H // kv
    o, mag, top = np.zeros_like(q), np.zeros_like(q), np.zeros((T, H))
    for i in range(len(cu) - 1):
        a, w = int(cu[i]), int(cu[i + 1] - cu[i])
        lim = np.repeat(int(lens[i]) - w + 1 + np.arange(w), G)
        for g in range(kv):
            pos, k, v = _keys(kc, vc, table[i], int(lens[i]), g, block)
            h = slice(g * G, (g + 1) * G)
            x, m, s = attend_rows(q[a:a + w, h].reshape(w * G, d), k, v, pos, lim, scale)
            o[a:a + w, h], mag[a:a + w, h] = x.reshape(w, G, d), m.reshape(w, G, d)
            top[a:a + w, h] = s.reshape(w, G)
    return o, mag, top


def shared_decode(q, k_cache, v_cache, table, lens, group_cu, prefix_lens, scale):
    """q [B, P, H, d]; the first prefix_lens[g] keys of a group's requests are those of the row of
    the first request that holds them all, or of the longest. Returns (o, mean |v|, absolute score
    sums [B, P, H])."""
    q, kc, vc = _f64(q), _f64(k_cache), _f64(v_cache)
    table, lens = _i32(table).copy(), _i32(lens)
    B, P, H, d = q.shape
    kv, block = kc.shape[1], kc.shape[2]
    G = H // kv
    first, skip = np.arange(B), np.zeros(B, dtype=np.int64)
    for g, x in enumerate(_i32(prefix_lens)):
        for b in range(int(group_cu[g]), int(group_cu[g + 1])):
            first[b], skip[b] = int(group_cu[g]), x
        rows = slice(int(group_cu[g]), int(group_cu[g + 1]))
        if rows.stop > rows.start:  # the first of those that hold the most of it
            first[rows] += int(np.argmax(np.clip(lens[rows], 0, x)))
    o, mag, top = np.zeros_like(q), np.zeros_like(q), np.zeros((B, P, H))
    for b in range(B):
        n = int(lens[b])
        lim = np.repeat(n - P + 1 + np.arange(P), G)
        for g in range(kv):
            head = _keys(kc, vc, table[first[b]], min(n, int(skip[b])), g, block)
            own = _keys(kc, vc, table[b], n, g, block)
            behind = own[0] >= skip[b]
            pos, k, v = (np.concatenate([x, y[behind]]) for x, y in zip(head, own))
            h = slice(g * G, (g + 1) * G)
            x, m, s = attend_rows(q[b, :, h].reshape(P * G, d), k, v, pos, lim, scale)
            o[b, :, h], mag[b, :, h] = x.reshape(P, G, d), m.reshape(P, G, d)
            top[b, :, h] = s.reshape(P, G)
    return o, mag, top
