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
