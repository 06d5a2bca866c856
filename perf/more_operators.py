"""Shared prefixes in the attention layers of a hybrid model's serving, case by case, for timing
and checking.

Requests of a serving engine often begin alike: samples and beams of one prompt, chats behind one
system prompt, questions about one document. Their tokens are then held once. The operators here
manage such pages and attend over them:

  fork           requests that continue others: their whole pages shared, the page that they will
                 write into copied, in every layer's cache
  free           requests that end: references dropped, pages that nobody holds any more listed
  compact        live pages moved to the front of the pool, in every layer's cache
  shared_decode  one token (or the P tokens of a verify step) per request, grouped heads, the
                 prefix that a group of requests shares read once for all of them
  prefill        a packed batch of prompts over the paged key/value cache, grouped heads, causal:
                 whole prompts, chunks of them, turns behind a cached (shared) prefix

`listed()` and `draw()` give cases, `prepare()` makes what a serving program has in hand before
the call, `run()` makes one pass: with `own` false in elementary torch operations, with `own`
true through this package's entry points. `exact()` evaluates the definitions in 64 bits.

`shares[page]` counts the holders of a page beyond the first, so 0 for pages of one request and
for free ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a beam search step: four beams continue one request, one layer
        dict(name="fork_beams", op="fork", parents=1, children=4, part=False, lens_lo=1000,
             lens_hi=1000, block=64, layers=1, heads=4, d=128, dtype="bf16"),
        # eight samples of each of many prompts, cut at any length; the caches of four layers
        dict(name="fork_samples", op="fork", parents=32, children=8, part=True, lens_lo=100,
             lens_hi=20000, block=64, layers=4, heads=4, d=128, dtype="bf16"),
        # one request ends
        dict(name="free_one", op="free", rows=48, n=1, lens_lo=900, lens_hi=9000, shared=0,
             block=64, pool=9000),
        # a large batch of samples ends, most of them behind shared prefixes; small pages
        dict(name="free_batch", op="free", rows=640, n=256, lens_lo=30, lens_hi=30000, shared=100,
             block=16, pool=300000),
        # a small pool before a long prompt is let in
        dict(name="compact_few", op="compact", rows=10, lens_lo=10, lens_hi=2000, shared=2,
             block=24, pool=600, layers=1, heads=2, d=64, dtype="f32"),
        # a pool that has been in use for long: four tenths of its pages live, spread all over
        dict(name="compact_pool", op="compact", rows=120, lens_lo=100, lens_hi=16000, shared=20,
             block=32, pool=29000, layers=2, heads=2, d=128, dtype="bf16"),
        # the smallest calls: two short prompts' samples, fp32, an odd page size
        dict(name="shared_few", op="shared_decode", dtype="f32", n=7, groups=2, loose=1, pos=1,
             heads=8, kv_heads=4, d=64, prefix_lo=90, prefix_hi=700, lens_lo=1, lens_hi=60,
             block=24),
        # a full serving batch behind one long document
        dict(name="shared_batch", op="shared_decode", dtype="bf16", n=128, groups=1, loose=0,
             pos=1, heads=32, kv_heads=4, d=128, prefix_lo=32000, prefix_hi=32000, lens_lo=30,
             lens_hi=2000, block=64),
        # the verify step of speculative decoding, wide heads, many small groups
        dict(name="shared_verify", op="shared_decode", dtype="bf16", n=48, groups=8, loose=4,
             pos=4, heads=16, kv_heads=2, d=256, prefix_lo=500, prefix_hi=16000, lens_lo=5,
             lens_hi=3000, block=32),
        # a few short turns, fp32
        dict(name="prompt_few", op="prefill", dtype="f32", n=3, heads=8, kv_heads=4, d=64,
             ctx_lo=1, ctx_hi=300, new_lo=5, new_hi=200, block=24),
        # one long prompt
        dict(name="prompt_long", op="prefill", dtype="bf16", n=1, heads=32, kv_heads=8, d=128,
             ctx_lo=0, ctx_hi=0, new_lo=12000, new_hi=12000, block=64),
        # a step of many turns, half of them behind a cached prefix
        dict(name="prompts_ragged", op="prefill", dtype="bf16", n=24, heads=32, kv_heads=4, d=128,
             ctx_lo=1, ctx_hi=16000, new_lo=3, new_hi=1500, block=32),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _lens(case, field, n):
    """n lengths of the case's range, the longest and the shortest among them. A range that
    starts at 1 in `ctx` stands for prefixes, and every other request there has none."""
    lo, hi = case[field + "_lo"], case[field + "_hi"]
    rng = random.Random("%s %s %s %s" % (field, lo, hi, n))
    out = [_spread(rng, max(lo, 1), hi) if hi else 0 for _ in range(n)]
    out[0] = hi
    if n > 1:
        out[-1] = lo
    if field == "ctx" and lo == 1:
        out = [0 if i % 2 else v for i, v in enumerate(out)]
    return out


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["op"], [0, 0])
        t[0], t[1] = max(t[0], w["bytes"]), max(t[1], w["flops"])
    op = rng.choice(sorted(top))
    block = rng.choice([8, 16, 20, 32, 64, 64, 128, 256, 640])
    if op == "fork":
        hi = _spread(rng, 10, 20000)
        c = dict(op=op, parents=_spread(rng, 1, 40), children=_spread(rng, 1, 16),
                 part=rng.choice([False, True]), lens_lo=_spread(rng, 1, hi), lens_hi=hi,
                 block=block, layers=rng.choice([1, 2, 4]), heads=rng.choice([1, 2, 3, 4]),
                 d=rng.choice([64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    elif op in ("free", "compact"):
        hi = _spread(rng, 10, 30000 if op == "free" else 16000)
        c = dict(op=op, rows=_spread(rng, 2, 600 if op == "free" else 300), lens_lo=1,
                 lens_hi=hi, block=block)
        c["shared"] = rng.choice([0, hi // (2 * block)])
        used = _live(c) + 1
        if op == "free":
            c["n"] = _spread(rng, 1, c["rows"])
            c["pool"] = min(_spread(rng, used, 4 * used), max(used, 300000))
        else:
            c["pool"] = _spread(rng, used, 4 * used)
            c.update(layers=rng.choice([1, 2]), heads=rng.choice([1, 2, 4]),
                     d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    elif op == "shared_decode":
        kv, group = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16])
        n = _spread(rng, 1, 150)
        groups = _spread(rng, 1, max(1, n // 2))
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), n=n, groups=groups,
                 loose=rng.choice([0, min(2, n - groups)]), pos=rng.choice([1, 1, 2, 3, 5]),
                 heads=kv * group, kv_heads=kv, d=rng.choice([64, 128, 256]), prefix_lo=1,
                 prefix_hi=_spread(rng, 10, 60000), lens_lo=5, lens_hi=_spread(rng, 10, 4000),
                 block=block)
    else:
        kv, group = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16])
        ctx_lo, ctx_hi = rng.choice([(0, 0), (1, _spread(rng, 10, 16000))])
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), n=_spread(rng, 1, 40),
                 heads=kv * group, kv_heads=kv, d=rng.choice([64, 128, 256]), ctx_lo=ctx_lo,
                 ctx_hi=ctx_hi, new_lo=1, new_hi=_spread(rng, 10, 12000), block=block)
    # (an fp32 product costs ten times a bf16 one)
    dear = 10 if c.get("dtype") == "f32" else 1
    while True:
        w = work(c)
        if w["bytes"] <= top[op][0] and w["flops"] * dear <= top[op][1]:
            return c
        for f in ("new_hi", "ctx_hi", "prefix_hi", "lens_hi", "pos", "parents", "children", "rows"):
            if f in c and (f != "rows" or op == "compact"):
                c[f] = max(1, c[f] // 2)
                lo = f.replace("_hi", "_lo")
                if lo != f:
                    c[lo] = min(c[lo], c[f])
        if op == "compact":
            c["shared"] = min(c["shared"], c["lens_hi"] // (2 * block))
            c["pool"] = 2 * _live(c) + 1


def _page(case):
    """Bytes of a page of one cache, and the number of caches."""
    e = 2 if case["dtype"] == "bf16" else 4
    return case["heads"] * case["block"] * case["d"] * e, 2 * case["layers"]


def _held(case):
    """Of the rows of a free or compact case: (pages, how many of them every second row shares
    with the row before it)."""
    out = []
    for i, x in enumerate(_lens(case, "lens", case["rows"])):
        need = -(-x // case["block"])
        common = min(case["shared"], x // case["block"], out[-1][0] if i % 2 else 0)
        out.append((need, common if i % 2 else 0))
    return out


def _live(case):
    return sum(a - b for a, b in _held(case))


def _forks(case):
    """(parent, length) of each fork."""
    lens = _lens(case, "lens", case["parents"])
    rng = random.Random(str(sorted(case.items())))
    return lens, [(p, rng.randint(1, lens[p]) if case["part"] else lens[p])
                  for p in range(case["parents"]) for _ in range(case["children"])]


def _groups(case):
    """(sizes, prefix lengths: whole pages) of the groups; `loose` requests come after them."""
    n, k = case["n"] - case["loose"], case["groups"]
    sizes = [n // k + (1 if i < n % k else 0) for i in range(k)]
    return sizes, [x // case["block"] * case["block"] for x in _lens(case, "prefix", k)]


def work(case):
    op, bs = case["op"], case["block"]
    if op == "fork":
        page, caches = _page(case)
        _, forks = _forks(case)
        whole = sum(x // bs for _, x in forks)
        copies = sum(x % bs > 0 for _, x in forks)
        # entries read and entered; shares of the pages read and written; source, destination and
        # length of a fork; ids taken and the pages copied
        return {"bytes": 16 * whole + 12 * len(forks) + copies * (16 + 2 * page * caches),
                "flops": 0}
    if op == "free":
        held = _held(case)
        gone = sum(a for a, _ in _freed_rows(case, held))
        # entries read and dropped, shares read and written, ids listed
        return {"bytes": 8 * case["n"] + gone * 20, "flops": 0}
    if op == "compact":
        page, caches = _page(case)
        held = _held(case)
        live, n = _live(case), case["pool"]
        moves = live * (n - live) // n  # of a random placement, on average
        entries = sum(a for a, _ in held)
        return {"bytes": 8 * entries + 4 * case["rows"] + moves * (24 + 2 * page * caches),
                "flops": 0}
    H, d, kv = case["heads"], case["d"], case["kv_heads"]
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["n"]
    if op == "shared_decode":
        sizes, prefix = _groups(case)
        mine, rows = sum(_lens(case, "lens", n)), n * case["pos"]
        seen = sum(s * p for s, p in zip(sizes, prefix)) + mine
        return {"bytes": (sum(prefix) + mine) * kv * 2 * d * e + 2 * rows * H * d * e,
                "flops": 4 * seen * case["pos"] * H * d}
    ctx, new = _lens(case, "ctx", n), _lens(case, "new", n)
    pairs = sum(c * w + w * (w + 1) // 2 for c, w in zip(ctx, new))
    return {"bytes": (sum(ctx) + sum(new)) * kv * 2 * d * e + 2 * sum(new) * H * d * e,
            "flops": 4 * pairs * H * d}


def _freed_rows(case, held):
    """The rows that end, spread over the table."""
    return [held[i * case["rows"] // case["n"]] for i in range(case["n"])]


# ----------------------------------------------------------------------------------- inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    """Inputs of one call, from the seed alone: values, page order, and which request has which
    of the case's lengths."""
    rng = random.Random(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, bs = case["op"], case["block"]

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)

    def caches(n_blocks):
        return [normal(n_blocks, case["heads"], bs, case["d"], dtype=TYPES[case["dtype"]])
                for _ in range(2 * case["layers"])]

    st = {"case": case, "op": op, "block": bs}
    if op == "fork":
        lens, forks = _forks(case)
        rng.shuffle(forks)
        need = [-(-x // bs) for x in lens]
        n_blocks = sum(need) + len(forks) + 5
        ids = list(range(n_blocks))
        rng.shuffle(ids)
        rows = len(lens) + len(forks)
        place = list(range(rows))  # table rows of the parents, then of their children
        rng.shuffle(place)
        table = [[-1] * (max(need) + 1) for _ in range(rows)]
        at = 0
        for i, k in enumerate(need):
            table[place[i]][:k] = ids[at:at + k]
            at += k
        st.update(src=_ints([place[p] for p, _ in forks]), lens=_ints([x for _, x in forks]),
                  dst=_ints(place[len(lens):]), table=_ints(table), free=_ints(ids[at:]),
                  shares=torch.zeros(n_blocks, dtype=torch.int32, device=DEV),
                  caches=caches(n_blocks))
        return st
    if op in ("free", "compact"):
        lens, held = _lens(case, "lens", case["rows"]), _held(case)
        ids = rng.sample(range(case["pool"]), _live(case))
        width = max(a for a, _ in held) + 1
        shares, table, at = [0] * case["pool"], [], 0
        for i, (need, common) in enumerate(held):
            row = table[-1][:common] if common else []
            for p in row:
                shares[p] += 1
            row = row + ids[at:at + need - common]
            at += need - common
            table.append(row + [-1] * (width - len(row)))
        order = list(range(len(lens)))
        rng.shuffle(order)
        st.update(table=_ints([table[i] for i in order]), shares=_ints(shares))
        if op == "compact":
            most = min(_live(case), case["pool"] - _live(case))
            st.update(lens=_ints([lens[i] for i in order]), most=most,
                      caches=caches(case["pool"]))
            return st
        back = {x: i for i, x in enumerate(order)}
        gone = [back[i * case["rows"] // case["n"]] for i in range(case["n"])]
        rng.shuffle(gone)
        st.update(rows=_ints(gone), lens=_ints([lens[order[i]] for i in gone]),
                  most=sum(-(-lens[order[i]] // bs) for i in gone))
        return st

    n, H, d, kv, dt = (case["n"], case["heads"], case["d"], case["kv_heads"],
                       TYPES[case["dtype"]])
    if op == "shared_decode":
        sizes, prefix = _groups(case)
        both = list(zip(sizes, prefix))
        rng.shuffle(both)
        mine = _lens(case, "lens", n)
        rng.shuffle(mine)
        cu, first = [0], []  # group bounds; shared tokens of each request
        for size, p in both:
            cu.append(cu[-1] + size)
            first += [p] * size
        first += [0] * case["loose"]
        lens = [a + b for a, b in zip(first, mine)]
        group = [g for g, (size, _) in enumerate(both) for _ in range(size)]
        group += [-1] * case["loose"]
        rows = (n, case["pos"])
        st.update(cu=_ints(cu), prefix=_ints([p for _, p in both]), host_cu=cu,
                  host_prefix=[p for _, p in both], host_lens=lens, host_first=first)
    else:
        ctx, new = _lens(case, "ctx", n), _lens(case, "new", n)
        order = list(range(n))
        rng.shuffle(order)
        lens, new = [ctx[i] + new[i] for i in order], [new[i] for i in order]
        cu = [0]
        for w in new:
            cu.append(cu[-1] + w)
        first, group, rows = [0] * n, [-1] * n, (cu[-1],)
        st.update(cu=_ints(cu), host_cu=cu, host_lens=lens)
    need = [-(-x // bs) - p // bs for x, p in zip(lens, first)]
    heads = {g: p // bs for g, p in zip(group, first) if g >= 0}
    n_blocks = sum(need) + sum(heads.values()) + 3
    ids = list(range(n_blocks))
    rng.shuffle(ids)
    at, common = 0, {-1: []}
    for g, k in heads.items():
        common[g] = ids[at:at + k]
        at += k
    width, table = max(max(-(-x // bs) for x in lens), 1), []
    for g, k in zip(group, need):
        row = common[g] + ids[at:at + k]
        at += k
        table.append(row + [-1] * (width - len(row)))
    # queries twice as long as keys: a softmax that singles out some of the keys
    st.update(table=_ints(table), lens=_ints(lens), scale=d ** -0.5,
              q=normal(*rows, H, d, scale=2.0, dtype=dt),
              k_cache=normal(n_blocks, kv, bs, d, dtype=dt),
              v_cache=normal(n_blocks, kv, bs, d, dtype=dt),
              o=torch.empty(*rows, H, d, dtype=dt, device=DEV))
    if own:
        from gated_delta_rule_prefill_amd import gdn
        if op == "shared_decode":
            size = gdn.gdn_paged_shared_decode_workspace_bytes(H, kv, d, dt, n, case["pos"],
                                                               case["groups"])
        else:
            size = gdn.gdn_paged_prefill_workspace_bytes(H, kv, d, dt, n, rows[0])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st


# --------------------------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _own_fork(s):
    from gated_delta_rule_prefill_amd import gdn
    out = gdn.gdn_paged_fork(s["src"], s["dst"], s["lens"], s["table"], s["block"], s["shares"],
                             s["free"])
    gdn.gdn_paged_copy(s["caches"], out[0], out[1])
    return [s["table"], s["shares"], *out, *s["caches"]]


# a request ends once: each pass takes the table as it was before
def _own_free(s):
    from gated_delta_rule_prefill_amd import gdn
    table, shares = s["table"].clone(), s["shares"].clone()
    out = gdn.gdn_paged_free(s["rows"], s["lens"], table, s["block"], shares,
                             max_freed=s["most"])
    return [table, shares, *out]


def _own_compact(s):
    from gated_delta_rule_prefill_amd import gdn
    table, shares = s["table"].clone(), s["shares"].clone()
    src, dst, counts = gdn.gdn_paged_compact(s["lens"], table, s["block"], shares,
                                             max_copies=s["most"])
    gdn.gdn_paged_copy(s["caches"], src, dst, count=counts[1:])
    return [table, shares, src, dst, counts, *s["caches"]]


def _own_shared_decode(s):
    from gated_delta_rule_prefill_amd import gdn
    return gdn.gdn_paged_shared_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                       s["cu"], s["prefix"], scale=s["scale"], o=s["o"],
                                       workspace=s["ws"])


def _own_prefill(s):
    from gated_delta_rule_prefill_amd import gdn
    return gdn.gdn_paged_prefill(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"],
                                 s["lens"], scale=s["scale"], o=s["o"], workspace=s["ws"])


_own = {"fork": _own_fork, "free": _own_free, "compact": _own_compact,
        "shared_decode": _own_shared_decode, "prefill": _own_prefill}


# the plain forms ---------------------------------------------------------------------------
def _copy_pages(caches, src, dst):
    real = (src >= 0).nonzero().flatten()
    a, b = src[real].long(), dst[real].long()
    for c in caches:
        c[b] = c[a]


def _plain_fork(s):
    src, dst, lens, table, bs = s["src"].long(), s["dst"].long(), s["lens"], s["table"], s["block"]
    whole = lens // bs
    col = torch.arange(table.shape[1], device=DEV)
    shared = col[None, :] < whole[:, None]
    from_row = table[src]
    rows = torch.where(shared, from_row, table[dst])
    count = (shared & (from_row >= 0)).to(torch.int32)
    s["shares"].index_add_(0, from_row.clamp_min(0).flatten(), count.flatten())
    last = from_row.gather(1, whole[:, None].long()).flatten()
    part = (lens % bs > 0) & (last >= 0)
    rank = part.cumsum(0) - 1
    fresh = torch.where(part & (rank < s["free"].numel()),
                        s["free"][rank.clamp(0, s["free"].numel() - 1)], -1)
    at = (lens % bs > 0)[:, None] & (col[None, :] == whole[:, None])
    table[dst] = torch.where(at, fresh[:, None], rows)
    copy_src = torch.where(fresh >= 0, last, -1)
    counts = torch.stack([part.sum(), (fresh >= 0).sum()]).to(torch.int32)
    _copy_pages(s["caches"], copy_src, fresh)
    return [table, s["shares"], copy_src, fresh, counts, *s["caches"]]


def _plain_free(s):
    table, shares, bs = s["table"].clone(), s["shares"].clone(), s["block"]
    rows = s["rows"].long()
    drop = torch.arange(table.shape[1], device=DEV) < ((s["lens"] + bs - 1) // bs)[:, None]
    pages = table[rows]
    held = drop & (pages >= 0)
    shares.index_add_(0, pages.clamp_min(0).flatten(), -held.to(torch.int32).flatten())
    table[rows] = torch.where(drop, -1, pages)
    gone = shares < 0
    shares.clamp_min_(0)
    freed = torch.full((s["most"] + 1,), -1, dtype=torch.int32, device=DEV)
    at = torch.where(gone, gone.cumsum(0) - 1, s["most"]).clamp_max(s["most"])
    freed[at] = torch.arange(shares.numel(), dtype=torch.int32, device=DEV)
    return [table, shares, freed[:-1], gone.sum().to(torch.int32).view(1)]


def _plain_compact(s):
    table, shares, bs, most = s["table"].clone(), s["shares"].clone(), s["block"], s["most"]
    n = shares.numel()
    held = torch.arange(table.shape[1], device=DEV) < ((s["lens"] + bs - 1) // bs)[:, None]
    held &= table >= 0
    live = torch.zeros(n + 1, dtype=torch.bool, device=DEV)
    live[torch.where(held, table, n).flatten().long()] = True
    live = live[:n]
    total = live.sum()
    ids = torch.arange(n, dtype=torch.int32, device=DEV)
    mover, hole = live & (ids >= total), ~live & (ids < total)
    pair = []
    for mask in (mover, hole):
        out = torch.full((most + 1,), -1, dtype=torch.int32, device=DEV)
        out[torch.where(mask, mask.cumsum(0) - 1, most).clamp_max(most)] = ids
        out[most] = -1
        pair.append(out[:most])
    src, dst = pair
    real = (src >= 0).nonzero().flatten()
    a, b = src[real].long(), dst[real].long()
    to = ids.clone()
    to[a] = dst[real]
    table = torch.where(held, to[table.clamp_min(0).long()], table)
    shares[b] = shares[a]
    shares[a] = 0
    for c in s["caches"]:
        c[b] = c[a]
    counts = torch.stack([total, mover.sum()]).to(torch.int32)
    return [table, shares, src, dst, counts, *s["caches"]]


def _rows_of(cache, table, n_tokens, bs):
    """Cache rows [requests, kv_heads, tokens, d] of the first tokens of table rows, fp32."""
    nb = -(-n_tokens // bs)
    x = cache[table[:, :nb].clamp_min(0).long()].permute(0, 2, 1, 3, 4)
    return x.reshape(table.shape[0], x.shape[1], nb * bs, x.shape[4]).float()


def _softmax(scores, keep):
    """Weights over the kept scores (unnormalised) and their sum, 1 where a row keeps none."""
    scores = scores.masked_fill_(~keep, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    e = scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = e.sum(dim=-1, keepdim=True)
    return e, torch.where(total == 0, torch.ones_like(total), total)


def _plain_shared_decode(s):
    """The prefix's scores and values in one product for a group, the requests' own in a batch."""
    q, bs, lens = s["q"], s["block"], s["lens"]
    n, P, H, d = q.shape
    kv = s["k_cache"].shape[1]
    G = H // kv
    out = torch.empty_like(q)
    runs = list(zip(s["host_cu"], s["host_cu"][1:], s["host_prefix"]))
    runs += [(i, i + 1, 0) for i in range(s["host_cu"][-1], n)]
    for a, z, shared in runs:
        b, skip = z - a, shared // bs
        longest = max(s["host_lens"][a:z]) - shared
        k, v = (_rows_of(c, s["table"][a:z, skip:], longest, bs)
                for c in (s["k_cache"], s["v_cache"]))
        x = q[a:z].float().view(b, P, kv, G, d).transpose(1, 2).reshape(b, kv, P * G, d)
        one = x.transpose(0, 1).reshape(kv, b * P * G, d)
        kp, vp = (_rows_of(c, s["table"][a:a + 1], shared, bs)[0] if shared else
                  k.new_zeros(kv, 0, d) for c in (s["k_cache"], s["v_cache"]))
        left = (one @ kp.transpose(1, 2)).view(kv, b, P * G, -1).transpose(0, 1)
        scores = torch.cat([left, x @ k.transpose(2, 3)], dim=3) * s["scale"]
        seen = (lens[a:z, None] - P + 1 + torch.arange(P, device=DEV)).repeat_interleave(G, dim=1)
        keep = torch.arange(scores.shape[3], device=DEV) < seen[:, None, :, None]
        e, total = _softmax(scores, keep)
        o = (e[..., :shared].transpose(0, 1).reshape(kv, b * P * G, shared) @ vp)
        o = o.view(kv, b, P * G, d).transpose(0, 1) + e[..., shared:] @ v
        out[a:z] = (o / total).view(b, kv, P, G, d).transpose(1, 2).reshape(b, P, H, d).to(q.dtype)
    return out


def _plain_prefill(s):
    q, bs = s["q"], s["block"]
    T, H, d = q.shape
    kv = s["k_cache"].shape[1]
    G = H // kv
    out = torch.empty_like(q)
    for i, L in enumerate(s["host_lens"]):
        a, z = s["host_cu"][i], s["host_cu"][i + 1]
        w = z - a
        k, v = (_rows_of(c, s["table"][i:i + 1], L, bs)[0, :, :L]
                for c in (s["k_cache"], s["v_cache"]))
        x = q[a:z].float().view(w, kv, G, d).permute(1, 2, 0, 3)
        keep = torch.arange(L, device=DEV) <= torch.arange(L - w, L, device=DEV)[:, None]
        step = max(1, min(kv, 2 ** 29 // max(1, w * L * G)))
        for h in range(0, kv, step):
            y = x[h:h + step].reshape(-1, G * w, d)
            scores = (y @ k[h:h + step].transpose(1, 2)).view(-1, G, w, L).mul_(s["scale"])
            e, total = _softmax(scores, keep)
            o = (e.view(-1, G * w, L) @ v[h:h + step]).view(-1, G, w, d) / total
            out[a:z, h * G:(h + o.shape[0]) * G] = o.reshape(-1, w, d).transpose(0, 1).to(q.dtype)
    return out


_plain = {"fork": _plain_fork, "free": _plain_free, "compact": _plain_compact,
          "shared_decode": _plain_shared_decode, "prefill": _plain_prefill}


# ------------------------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact[s["op"]](s)


def _moved(caches, pairs):
    """Each cache after its pages are copied, one pair after another."""
    out = []
    for c in caches:
        x = c.double()
        for a, b in pairs:
            x[b].copy_(x[a])
        out.append(x)
    return out


def _exact_fork(s):
    """One fork after another, one page after another."""
    table, free, shares, bs = s["table"].tolist(), s["free"].tolist(), s["shares"].tolist(), s["block"]
    pairs, asked = [], 0
    for src, dst, x in zip(s["src"].tolist(), s["dst"].tolist(), s["lens"].tolist()):
        for p in range(x // bs):
            table[dst][p] = table[src][p]
            shares[table[src][p]] += 1
        pair = (-1, -1)
        if x % bs:
            pair = (table[src][x // bs], free[asked])
            table[dst][x // bs] = free[asked]
            asked += 1
        pairs.append(pair)
    real = [p for p in pairs if p[0] >= 0]
    return [_ints(table), _ints(shares), _ints([p[0] for p in pairs]), _ints([p[1] for p in pairs]),
            _ints([asked, len(real)]), *_moved(s["caches"], real)]


def _exact_free(s):
    table, shares, bs = s["table"].tolist(), s["shares"].tolist(), s["block"]
    gone = []
    for row, x in zip(s["rows"].tolist(), s["lens"].tolist()):
        for p in range(-(-x // bs)):
            page, table[row][p] = table[row][p], -1
            if shares[page]:
                shares[page] -= 1
            else:
                gone.append(page)
    freed = sorted(gone) + [-1] * (s["most"] - len(gone))
    return [_ints(table), _ints(shares), _ints(freed), _ints([len(gone)])]


def _exact_compact(s):
    table, shares, bs = s["table"].tolist(), s["shares"].tolist(), s["block"]
    lens = s["lens"].tolist()
    live = sorted({p for row, x in zip(table, lens) for p in row[:-(-x // bs)]})
    src = [p for p in live if p >= len(live)]
    dst = sorted(set(range(len(live))) - set(live))
    to = dict(zip(src, dst))
    for row, x in zip(table, lens):
        for p in range(-(-x // bs)):
            row[p] = to.get(row[p], row[p])
    for a, b in to.items():
        shares[a], shares[b] = 0, shares[a]
    pad = [-1] * (s["most"] - len(src))
    return [_ints(table), _ints(shares), _ints(src + pad), _ints(dst + pad),
            _ints([len(live), len(src)]), *_moved(s["caches"], to.items())]


def _exact_attend(q, k, v, first, scale):
    """q [h, t, d] against k, v [L, d] in 64 bits; row i sees keys 0 .. first + i."""
    x = torch.matmul(k, q.transpose(1, 2)).mul_(scale)          # [h, L, t]
    seen = first + torch.arange(q.shape[1], device=DEV)
    x.masked_fill_(torch.arange(k.shape[0], device=DEV)[:, None] > seen[None, :], -math.inf)
    p = torch.softmax(x, dim=1).nan_to_num_(0.0)  # a row without keys gives zeros
    return torch.matmul(p.transpose(1, 2), v)


def _exact_request(s, q, i, L):
    """q [t, H, d]: the newest t tokens of request i, keys taken from its own table row."""
    t, H, d = q.shape
    kv, bs = s["k_cache"].shape[1], s["block"]
    ids = s["table"][i, :-(-L // bs)].long()
    out = torch.empty_like(q)
    step = max(1, 2 ** 28 // max(1, L * t))
    for g in range(kv):
        k = s["k_cache"][ids, g].reshape(-1, d)[:L].double()
        v = s["v_cache"][ids, g].reshape(-1, d)[:L].double()
        for h in range(g * (H // kv), (g + 1) * (H // kv), step):
            e = min(h + step, (g + 1) * (H // kv))
            o = _exact_attend(q[:, h:e].transpose(0, 1), k, v, L - t, s["scale"])
            out[:, h:e] = o.transpose(0, 1)
    return out


def _exact_shared_decode(s):
    q = s["q"].double()
    return torch.stack([_exact_request(s, q[i], i, L) for i, L in enumerate(s["host_lens"])])


def _exact_prefill(s):
    q, cu = s["q"].double(), s["host_cu"]
    return torch.cat([_exact_request(s, q[cu[i]:cu[i + 1]], i, L)
                      for i, L in enumerate(s["host_lens"])])


_exact = {"fork": _exact_fork, "free": _exact_free, "compact": _exact_compact,
          "shared_decode": _exact_shared_decode, "prefill": _exact_prefill}
