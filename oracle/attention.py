"""fp64 numpy reference of the paged softmax-attention operators: block tables and slot maps,
cache rows, attention over pages, and the two forms of latent attention.

Plain loops over requests and positions, from the definitions. Every attention function also
returns what a tolerance needs: for each output the mean of |v| under its weights, and for each
query the largest sum of |q_i k_i| of a score (both bound what a rounded operand can move).
"""
import numpy as np

from . import _f64, _i32


def plan(ctx, new, table, free, block, max_tokens):
    """One request after another, one token after another. Returns (table, cu, lens, slots,
    positions, counts)."""
    table = _i32(table).copy()
    free = [int(x) for x in _i32(free)]
    n, width = table.shape
    cu, lens, slots, positions, asked, total = [0], [], [], [], 0, 0
    for i in range(n):
        c, w = max(int(ctx[i]), 0), max(int(new[i]), 0)
        held = -(-c // block)
        for p in range(c, c + w):
            page, off = p // block, p % block
            if page >= width:
                slot = -1
            else:
                if page >= held and off == 0:
                    got = free[asked] if asked < len(free) else -1
                    asked += 1
                    if total < max_tokens:
                        table[i, page] = got
                blk = int(table[i, page])
                slot = blk * block + off if blk >= 0 else -1
            if total < max_tokens:
                slots.append(slot)
                positions.append(p)
            total += 1
        cu.append(total)
        lens.append(c + w)
    pad = max_tokens - len(slots)
    return (table, np.array(cu), np.array(lens), np.array(slots + [-1] * pad, dtype=np.int64),
            np.array(positions + [0] * pad), np.array([total, asked]))


def visible(table_row, n_tokens, block, n_blocks):
    """(position, page, offset) of the tokens that exist among the first n_tokens."""
    out = []
    for j in range(min(max(n_tokens, 0), len(table_row) * block)):
        page = int(table_row[j // block])
        if 0 <= page < n_blocks:
            out.append((j, page, j % block))
    return out


def attend(q, k, v, scale):
    """One query over the given keys: (output, mean |v| under the weights, largest absolute
    score sum). No keys: zeros."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), np.zeros(v.shape[1]), 0.0
    s = scale * (k @ q)
    e = np.exp(s - s.max())
    p = e / e.sum()
    return p @ v, p @ np.abs(v), float(np.max(abs(scale) * (np.abs(k) @ np.abs(q))))


def paged_decode(q, k_cache, v_cache, table, lens, scale):
    """q [B, P, H, d]; caches [n_blocks, kv_heads, block, d]. Returns (o, mean |v|, absolute
    score sums [B, P, H])."""
    q, kc, vc = _f64(q), _f64(k_cache), _f64(v_cache)
    table, lens = _i32(table), _i32(lens)
    B, P, H, d = q.shape
    n_blocks, kv, block, _ = kc.shape
    o, mag, top = np.zeros_like(q), np.zeros_like(q), np.zeros((B, P, H))
    for b in range(B):
        seen = visible(table[b], int(lens[b]), block, n_blocks)
        pos = np.array([x[0] for x in seen], dtype=np.int64)
        page = np.array([x[1] for x in seen], dtype=np.int64)
        off = np.array([x[2] for x in seen], dtype=np.int64)
        for g in range(kv):
            k, v = kc[page, g, off], vc[page, g, off]
            for p in range(P):
                m = pos < int(lens[b]) - P + p + 1
                for h in range(g * (H // kv), (g + 1) * (H // kv)):
                    o[b, p, h], mag[b, p, h], top[b, p, h] = attend(q[b, p, h], k[m], v[m], scale)
    return o, mag, top


def _latent_rows(cache, table_row, n_tokens):
    """Existing cache rows of one request: (their positions, the rows) in fp64."""
    n_blocks, block, _ = cache.shape
    seen = visible(table_row, n_tokens, block, n_blocks)
    pos = np.array([x[0] for x in seen], dtype=np.int64)
    rows = cache[[x[1] for x in seen], [x[2] for x in seen]] if seen else cache[0, :0]
    return pos, rows


def _weights(s):
    e = np.exp(s - s.max())
    return e / e.sum()


def latent_absorbed(q_nope, q_pe, w_kv, cache, table, lens, scale):
    """Queries taken into the latent space, outputs taken out of it; q_* [B, P, H, .]."""
    qn, qp, w, c = _f64(q_nope), _f64(q_pe), _f64(w_kv), _f64(cache)
    table, lens = _i32(table), _i32(lens)
    B, P, H, dn = qn.shape
    R = w.shape[2]
    o = np.zeros((B, P, H, w.shape[1] - dn))
    for b in range(B):
        pos, rows = _latent_rows(c, table[b], int(lens[b]))
        for p in range(P):
            x = rows[pos < int(lens[b]) - P + p + 1]
            if len(x) == 0:
                continue
            for h in range(H):
                q = np.concatenate([qn[b, p, h] @ w[h, :dn], qp[b, p, h]])
                o[b, p, h] = w[h, dn:] @ (_weights(scale * (x @ q)) @ x[:, :R])
    return o


def latent_expanded(q_nope, q_pe, w_kv, cache, table, cu, lens, scale):
    """Every head's keys and values written out; packed q_* [T, H, .], causal: the tokens of a
    request are its last cu[i + 1] - cu[i]."""
    qn, qp, w, c = _f64(q_nope), _f64(q_pe), _f64(w_kv), _f64(cache)
    table, lens, cu = _i32(table), _i32(lens), _i32(cu)
    T, H, dn = qn.shape
    R = w.shape[2]
    o = np.zeros((T, H, w.shape[1] - dn))
    for i in range(len(cu) - 1):
        pos, rows = _latent_rows(c, table[i], int(lens[i]))
        new = int(cu[i + 1] - cu[i])
        for h in range(H):
            k = np.concatenate([rows[:, :R] @ w[h, :dn].T, rows[:, R:]], axis=1)
            v = rows[:, :R] @ w[h, dn:].T
            for t in range(new):
                m = pos <= int(lens[i]) - new + t
                if not m.any():
                    continue
                q = np.concatenate([qn[cu[i] + t, h], qp[cu[i] + t, h]])
                o[cu[i] + t, h] = _weights(scale * (k[m] @ q)) @ v[m]
    return o


def latent_error(q_nope, q_pe, w_kv, rows, o, scale, u):
    """Standard deviations that independent roundings leave in one output, for a query (q_nope
    [dn], q_pe) of one head (w_kv [dn + dv, R]) over fp64 cache rows, with half step u: a
    rounding's error is at most u of the value, and spread evenly over that range u / sqrt(3) of
    it. Counted: the latent-space query (one rounding moves the scores of all keys together) and
    the written-out keys, each softmax weight, the mixed latent and the written-out values, the
    output. The absorbed and the expanded form make only some of these."""
    dn, R = q_nope.shape[0], w_kv.shape[1]
    if len(rows) == 0:
        return np.zeros(w_kv.shape[0] - dn)
    c = rows[:, :R]
    ql, k, v = q_nope @ w_kv[:dn], c @ w_kv[:dn].T, c @ w_kv[dn:].T
    p = _weights(scale * (c @ ql + rows[:, R:] @ q_pe))
    e = u / np.sqrt(3.0)
    dev = v - o                                   # a weight's error moves o by p_j (v_j - o)
    query = scale * e * np.sqrt(((ql[:, None] * ((p[:, None] * c).T @ dev)) ** 2).sum(0))
    key = scale * e * np.sqrt(((k * q_nope) ** 2).sum(1))
    from_scores = np.hypot(query, np.sqrt((((p * key)[:, None] * dev) ** 2).sum(0)))
    from_weights = e * np.sqrt(((p[:, None] * v) ** 2).sum(0))
    mixed = e * np.sqrt(np.maximum(((w_kv[dn:] * (p @ c)) ** 2).sum(1),
                                   ((p[:, None] * v) ** 2).sum(0)))
    return np.sqrt(from_scores ** 2 + from_weights ** 2 + mixed ** 2 + (e * o) ** 2)
