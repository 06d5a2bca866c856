"""The attention side of a hybrid model's serving step, case by case, for timing and checking.

A hybrid model interleaves gated delta-rule layers (one fixed-size state per request) with
softmax-attention layers, whose keys and values live in a paged cache. The operators here are
that second half:

  plan            block tables, slot maps, positions and cu_seqlens from request lengths
  append          new tokens' rows written to a paged key/value cache or latent cache
  paged_decode    one token (or the P tokens of a verify step) per request against a paged
                  key/value cache, grouped heads
  latent_decode   the same against a cache of one shared latent vector and one rotary key per
                  token, absorbed form
  latent_prefill  a packed batch of prompts against that cache, expanded form, causal

`listed()` and `draw()` give cases, `prepare()` makes what a serving program has in hand before
the call, `run()` makes one pass: with `own` false in elementary torch operations, with `own`
true through this package's entry points. `exact()` evaluates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
ROPE = 64  # width of the shared rotary key of a latent row
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's bookkeeping: 24 running requests get one token each
        dict(name="plan_step", op="plan", n=24, ctx_lo=100, ctx_hi=9000, new_lo=1, new_hi=1,
             block=64, pad=0),
        # a large prefill step: prompts of every length, some of them with a cached prefix, into
        # small pages; the token buffers are sized for the engine's step limit
        dict(name="plan_prompts", op="plan", n=320, ctx_lo=1, ctx_hi=3000, new_lo=1, new_hi=4000,
             block=16, pad=5000),
        # a decode step's rows of one layer into a key/value cache
        dict(name="append_step", op="append", form="kv", dtype="bf16", tokens=96, heads=4, d=128,
             block=64),
        # a prefill step's latents, read out of the projection's output in place
        dict(name="append_prompts", op="append", form="latent", dtype="bf16", tokens=65000,
             rank=512, block=64),
        # the smallest call: a few short requests, fp32, an odd page size
        dict(name="decode_few", op="paged_decode", dtype="f32", n=3, pos=1, heads=8, kv_heads=4,
             d=64, lens_lo=17, lens_hi=500, block=24),
        # one user with a long document
        dict(name="decode_long", op="paged_decode", dtype="bf16", n=1, pos=1, heads=32,
             kv_heads=8, d=128, lens_lo=250001, lens_hi=250001, block=64),
        # a full serving batch, lengths spread over three decades
        dict(name="decode_batch", op="paged_decode", dtype="bf16", n=128, pos=1, heads=32,
             kv_heads=4, d=128, lens_lo=30, lens_hi=30000, block=64),
        # the verify step of speculative decoding, wide heads
        dict(name="verify_batch", op="paged_decode", dtype="bf16", n=40, pos=4, heads=16,
             kv_heads=2, d=256, lens_lo=200, lens_hi=20000, block=32),
        # one request on a GPU that holds a share of the heads
        dict(name="latent_decode_one", op="latent_decode", n=1, pos=1, heads=20, rank=512, d=128,
             lens_lo=40003, lens_hi=40003, block=64),
        # a full serving batch with every head on the GPU
        dict(name="latent_decode_batch", op="latent_decode", n=80, pos=1, heads=128, rank=512,
             d=128, lens_lo=100, lens_hi=12000, block=64),
        # one prompt
        dict(name="latent_prompt", op="latent_prefill", n=1, heads=32, rank=512, d=128,
             ctx_lo=0, ctx_hi=0, new_lo=8192, new_hi=8192, block=64),
        # a step of many prompts, half of them resumed behind a cached prefix
        dict(name="latent_prompts", op="latent_prefill", n=28, heads=20, rank=512, d=128,
             ctx_lo=1, ctx_hi=6000, new_lo=3, new_hi=1500, block=64),
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
    if op == "plan":
        new_lo, new_hi = rng.choice([(1, 1), (0, 5), (1, _spread(rng, 2, 5000))])
        c = dict(op=op, n=_spread(rng, 1, 1000), ctx_lo=rng.choice([0, 1]),
                 ctx_hi=_spread(rng, 10, 50000), new_lo=new_lo, new_hi=new_hi, block=block,
                 pad=rng.choice([0, _spread(rng, 1, 5000)]))
        long = "new_hi"
    elif op == "append":
        c = dict(op=op, form=rng.choice(["kv", "latent"]), tokens=_spread(rng, 1, 65000),
                 block=block)
        if c["form"] == "kv":
            c.update(dtype=rng.choice(["bf16", "f32"]), heads=rng.choice([1, 2, 3, 4, 8]),
                     d=rng.choice([64, 128, 256]))
        else:
            c.update(dtype="bf16", rank=rng.choice([256, 512]))
        long = "tokens"
    elif op == "paged_decode":
        kv, group = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16])
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), n=_spread(rng, 1, 200),
                 pos=rng.choice([1, 1, 2, 3, 5]), heads=kv * group, kv_heads=kv,
                 d=rng.choice([64, 128, 256]), lens_lo=1,
                 lens_hi=_spread(rng, 10, 200000), block=block)
        long = "lens_hi"
    elif op == "latent_decode":
        c = dict(op=op, n=_spread(rng, 1, 150), pos=rng.choice([1, 1, 2, 4]),
                 heads=rng.choice([8, 16, 20, 32, 64, 128]), rank=rng.choice([256, 512, 512]),
                 d=rng.choice([64, 128, 128]), lens_lo=1,
                 lens_hi=_spread(rng, 10, 100000), block=block)
        long = "lens_hi"
    else:
        ctx_lo, ctx_hi = rng.choice([(0, 0), (1, _spread(rng, 10, 8000))])
        c = dict(op=op, n=_spread(rng, 1, 40), heads=rng.choice([5, 8, 16, 32, 64]),
                 rank=rng.choice([256, 512, 512]), d=rng.choice([64, 128, 128]),
                 ctx_lo=ctx_lo, ctx_hi=ctx_hi, new_lo=1, new_hi=_spread(rng, 10, 8000),
                 block=block)
        long = "new_hi"
    while True:
        w = work(c)
        if w["bytes"] <= top[op][0] and w["flops"] <= top[op][1]:
            return c
        for f in (long, "ctx_hi"):
            if f in c:
                c[f] = c[f] // 2
                c[f.replace("hi", "lo")] = min(c.get(f.replace("hi", "lo"), c[f]), c[f])


def work(case):
    op = case["op"]
    if op == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        row = 2 * case["heads"] * case["d"] if case["form"] == "kv" else case["rank"] + ROPE
        return {"bytes": case["tokens"] * (2 * row * e + 8), "flops": 0}
    n = case["n"]
    if op == "plan":
        ctx, new = _lens(case, "ctx", n), _lens(case, "new", n)
        held = [-(-c // case["block"]) for c in ctx]
        need = sum(-(-(c + w) // case["block"]) - h for c, w, h in zip(ctx, new, held))
        # lengths in; ids of the new blocks read and entered, the block that the first new token
        # of a request continues; cu_seqlens and lengths out; slot and position of each token
        b = 8 * n + 8 * need + 4 * n + 4 * (2 * n + 1) + 12 * (sum(new) + case["pad"]) + 8
        return {"bytes": b, "flops": 2 * n + 3 * sum(new)}
    H, d = case["heads"], case["d"]
    if op == "paged_decode":
        e = 2 if case["dtype"] == "bf16" else 4
        keys, rows = sum(_lens(case, "lens", n)), n * case["pos"]
        return {"bytes": keys * case["kv_heads"] * 2 * d * e + 2 * rows * H * d * e,
                "flops": 4 * keys * case["pos"] * H * d}
    R = case["rank"]
    weights = 2 * H * 2 * d * R
    if op == "latent_decode":
        keys, rows = sum(_lens(case, "lens", n)), n * case["pos"]
        return {"bytes": keys * (R + ROPE) * 2 + weights + rows * H * (2 * d + ROPE) * 2,
                "flops": 2 * keys * case["pos"] * H * (2 * R + ROPE) + 4 * rows * H * d * R}
    ctx, new = _lens(case, "ctx", n), _lens(case, "new", n)
    keys, rows = sum(ctx) + sum(new), sum(new)
    pairs = sum(c * w + w * (w + 1) // 2 for c, w in zip(ctx, new))
    return {"bytes": keys * (R + ROPE) * 2 + weights + rows * H * (2 * d + ROPE) * 2,
            "flops": 4 * keys * R * H * d + 2 * pairs * H * (2 * d + ROPE)}


# ----------------------------------------------------------------------------------- inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pages(rng, lens, block, spare):
    """Block ids for every request, in a random order of the pool, the table's free entries -1.
    Returns (table, ids of the free blocks, number of blocks)."""
    need = [-(-x // block) for x in lens]
    total = sum(need) + spare
    ids = list(range(total))
    rng.shuffle(ids)
    width = max(max(need), 1)
    rows, at = [], 0
    for k in need:
        rows.append(ids[at:at + k] + [-1] * (width - k))
        at += k
    return rows, ids[at:], total


def prepare(case, seed):
    """Inputs of one call, from the seed alone: values, page order, and which request has which
    of the case's lengths."""
    rng = random.Random(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, block = case["op"], case["block"]

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)

    st = {"case": case, "op": op, "block": block}
    if op == "append":
        T, dt = case["tokens"], TYPES[case["dtype"]]
        n_blocks = -(-T // block) + 5
        slots = torch.randperm(n_blocks * block, generator=gen, device=DEV)[:T].contiguous()
        st.update(slots=slots, n_blocks=n_blocks)
        if case["form"] == "kv":
            H, d = case["heads"], case["d"]
            qkv = normal(T, 3 * H, d, dtype=dt)  # one projection's output: q, k and v heads
            st.update(a=qkv[:, H:2 * H], b=qkv[:, 2 * H:],
                      cache_a=normal(n_blocks, H, block, d, dtype=dt),
                      cache_b=normal(n_blocks, H, block, d, dtype=dt))
        else:
            R = case["rank"]
            kv = normal(T, R + ROPE, dtype=dt)  # the down projection: latent and rotary key
            st.update(a=kv[:, :R], b=kv[:, R:], cache_a=normal(n_blocks, block, R + ROPE, dtype=dt))
        return st

    n = case["n"]
    order = list(range(n))
    rng.shuffle(order)
    if op == "plan":
        ctx, new = _lens(case, "ctx", n), _lens(case, "new", n)
        ctx, new = [ctx[i] for i in order], [new[i] for i in order]
        rows, _, total = _pages(rng, ctx, block, 0)
        width = max(-(-(c + w) // block) for c, w in zip(ctx, new)) + 1
        rows = [r[:width] + [-1] * (width - len(r)) for r in rows]
        need = sum(-(-(c + w) // block) - -(-c // block) for c, w in zip(ctx, new))
        free = list(range(total, total + need + 7))
        rng.shuffle(free)
        T = sum(new) + case["pad"]
        st.update(ctx=_ints(ctx), new=_ints(new), table=_ints(rows), free=_ints(free), tokens=T,
                  cu=torch.empty(n + 1, dtype=torch.int32, device=DEV),
                  lens=torch.empty(n, dtype=torch.int32, device=DEV),
                  slots=torch.empty(T, dtype=torch.int64, device=DEV),
                  positions=torch.empty(T, dtype=torch.int32, device=DEV),
                  counts=torch.empty(2, dtype=torch.int32, device=DEV))
        return st

    H, d = case["heads"], case["d"]
    if op == "latent_prefill":
        ctx, new = _lens(case, "ctx", n), _lens(case, "new", n)
        lens = [ctx[i] + new[i] for i in order]
        new = [new[i] for i in order]
        cu = [0]
        for w in new:
            cu.append(cu[-1] + w)
        st.update(cu=_ints(cu), host_cu=cu, keys=sum(lens))
    else:
        lens = _lens(case, "lens", n)
        lens = [lens[i] for i in order]
    rows, _, n_blocks = _pages(rng, lens, block, 3)
    st.update(table=_ints(rows), lens=_ints(lens), host_lens=lens)
    if op == "paged_decode":
        dt, P, kv = TYPES[case["dtype"]], case["pos"], case["kv_heads"]
        # queries twice as long as keys: a softmax that singles out some of the keys
        st.update(q=normal(n, P, H, d, scale=2.0, dtype=dt),
                  k_cache=normal(n_blocks, kv, block, d, dtype=dt),
                  v_cache=normal(n_blocks, kv, block, d, dtype=dt),
                  scale=d ** -0.5, o=torch.empty(n, P, H, d, dtype=dt, device=DEV))
        if own:
            from gated_delta_rule_prefill_amd import gdn
            st["ws"] = torch.empty(gdn.gdn_paged_decode_workspace_bytes(H, kv, d, dt, n, P),
                                   dtype=torch.uint8, device=DEV)
        return st
    R = case["rank"]
    rows = (st["host_cu"][-1],) if op == "latent_prefill" else (n, case["pos"])
    st.update(q_nope=normal(*rows, H, d, scale=1.5), q_pe=normal(*rows, H, ROPE, scale=1.5),
              w_kv=normal(H, 2 * d, R, scale=R ** -0.5),  # a trained up projection keeps the scale
              cache=normal(n_blocks, block, R + ROPE), scale=(d + ROPE) ** -0.5,
              o=torch.empty(*rows, H, d, dtype=torch.bfloat16, device=DEV))
    if own:
        from gated_delta_rule_prefill_amd import gdn
        if op == "latent_decode":
            size = gdn.gdn_latent_decode_workspace_bytes(H, R, ROPE, d, d, n, case["pos"])
        else:
            size = gdn.gdn_latent_prefill_workspace_bytes(H, R, ROPE, d, d, n, rows[0], st["keys"])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st


# --------------------------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _own_plan(s):
    from gated_delta_rule_prefill_amd import gdn
    out = gdn.gdn_paged_plan(s["ctx"], s["new"], s["table"], s["free"], s["block"], s["tokens"],
                             cu_seqlens=s["cu"], seq_lens=s["lens"], slot_map=s["slots"],
                             positions=s["positions"], counts=s["counts"])
    return [s["table"], *out]


def _own_append(s):
    from gated_delta_rule_prefill_amd import gdn
    if s["case"]["form"] == "kv":
        gdn.gdn_paged_append(s["a"], s["b"], s["slots"], s["cache_a"], s["cache_b"])
        return [s["cache_a"], s["cache_b"]]
    gdn.gdn_latent_append(s["a"], s["b"], s["slots"], s["cache_a"])
    return [s["cache_a"]]


def _own_paged_decode(s):
    from gated_delta_rule_prefill_amd import gdn
    return gdn.gdn_paged_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                scale=s["scale"], o=s["o"], workspace=s["ws"])


def _own_latent_decode(s):
    from gated_delta_rule_prefill_amd import gdn
    return gdn.gdn_latent_decode(s["q_nope"], s["q_pe"], s["w_kv"], s["cache"], s["table"],
                                 s["lens"], scale=s["scale"], o=s["o"], workspace=s["ws"])


def _own_latent_prefill(s):
    from gated_delta_rule_prefill_amd import gdn
    return gdn.gdn_latent_prefill(s["q_nope"], s["q_pe"], s["w_kv"], s["cache"], s["table"],
                                  s["cu"], s["lens"], s["keys"], scale=s["scale"], o=s["o"],
                                  workspace=s["ws"])


_own = {"plan": _own_plan, "append": _own_append, "paged_decode": _own_paged_decode,
        "latent_decode": _own_latent_decode, "latent_prefill": _own_latent_prefill}


# the plain forms ---------------------------------------------------------------------------
def _plain_plan(s):
    ctx, new, table, free = s["ctx"], s["new"], s["table"], s["free"]
    bs, T = s["block"], s["tokens"]
    n = ctx.numel()
    lens = ctx + new
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), new.cumsum(0).to(torch.int32)])
    held = (ctx + bs - 1) // bs
    need = (lens + bs - 1) // bs - held
    first = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    take = (first[:, None] + col - held[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[take], table))
    t = torch.arange(T, device=DEV)
    req = torch.searchsorted(cu[1:].long(), t, right=True).clamp_max(n - 1)
    live = t < cu[-1]
    pos = t - cu[req] + ctx[req]
    page = table[req, (pos // bs).clamp_max(table.shape[1] - 1)].long()
    slots = torch.where(live, page * bs + pos % bs, -1)
    positions = torch.where(live, pos, 0).to(torch.int32)
    counts = torch.stack([cu[-1], need.sum().to(torch.int32)])
    return [table, cu, lens, slots, positions, counts]


def _plain_append(s):
    slots, bs = s["slots"], s["block"]
    if s["case"]["form"] == "kv":
        page, at = slots // bs, slots % bs
        s["cache_a"][page, :, at] = s["a"]
        s["cache_b"][page, :, at] = s["b"]
        return [s["cache_a"], s["cache_b"]]
    s["cache_a"].view(-1, s["cache_a"].shape[2])[slots] = torch.cat([s["a"], s["b"]], dim=1)
    return [s["cache_a"]]


def _softmax_times(scores, keep, values):
    """softmax over the kept scores times values, zeros where a row keeps none."""
    scores = scores.masked_fill(~keep, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(dim=-1, keepdim=True)
    return (e @ values) / torch.where(total == 0, torch.ones_like(total), total)


def _slices(lens, floats_a_key, top=2 ** 28):
    """Runs of requests whose padded keys stay within `top` fp32 numbers."""
    at = 0
    while at < len(lens):
        end, longest = at + 1, lens[at]
        while end < len(lens) and (end + 1 - at) * max(longest, lens[end]) * floats_a_key <= top:
            longest = max(longest, lens[end])
            end += 1
        yield at, end, max(longest, 1)
        at = end


def _plain_paged_decode(s):
    q, bs, lens = s["q"], s["block"], s["lens"]
    n, P, H, d = q.shape
    kv = s["k_cache"].shape[1]
    G = H // kv
    out = torch.empty_like(q)
    for a, z, longest in _slices(s["host_lens"], kv * d):
        b, nb = z - a, -(-longest // bs)
        table = s["table"][a:z, :nb].clamp_min(0).long()
        k, v = (c[table].permute(0, 2, 1, 3, 4).reshape(b, kv, nb * bs, d).float()
                for c in (s["k_cache"], s["v_cache"]))
        qs = q[a:z].float().view(b, P, kv, G, d).transpose(1, 2).reshape(b, kv, P * G, d)
        scores = qs @ k.transpose(2, 3) * s["scale"]
        seen = lens[a:z, None] - P + 1 + torch.arange(P, device=DEV)
        seen = seen.repeat_interleave(G, dim=1)[:, None, :, None]
        keep = torch.arange(nb * bs, device=DEV) < seen
        o = _softmax_times(scores, keep, v)
        out[a:z] = o.view(b, kv, P, G, d).transpose(1, 2).reshape(b, P, H, d).to(q.dtype)
    return out


def _plain_latent_decode(s):
    qn, qp, w, bs, lens = s["q_nope"], s["q_pe"], s["w_kv"], s["block"], s["lens"]
    n, P, H, d = qn.shape
    R = w.shape[2]
    wf = w.float()
    lat = (qn.float().view(n * P, H, d).transpose(0, 1) @ wf[:, :d]).transpose(0, 1)
    q = torch.cat([lat.reshape(n, P * H, R), qp.float().view(n, P * H, ROPE)], dim=2)
    mixed = torch.empty(n, P * H, R, device=DEV)
    for a, z, longest in _slices(s["host_lens"], R + ROPE):
        b, nb = z - a, -(-longest // bs)
        table = s["table"][a:z, :nb].clamp_min(0).long()
        k = s["cache"][table].reshape(b, nb * bs, R + ROPE).float()
        scores = q[a:z] @ k.transpose(1, 2) * s["scale"]
        seen = lens[a:z, None] - P + 1 + torch.arange(P, device=DEV)
        keep = torch.arange(nb * bs, device=DEV) < seen.repeat_interleave(H, dim=1)[:, :, None]
        mixed[a:z] = _softmax_times(scores, keep, k[..., :R])
    o = mixed.view(n * P, H, R).transpose(0, 1) @ wf[:, d:].transpose(1, 2)
    return o.transpose(0, 1).reshape(n, P, H, d).to(qn.dtype)


def _plain_latent_prefill(s):
    qn, qp, w, bs = s["q_nope"], s["q_pe"], s["w_kv"], s["block"]
    T, H, d = qn.shape
    R = w.shape[2]
    out = torch.empty_like(qn)
    for i, L in enumerate(s["host_lens"]):
        a, z = s["host_cu"][i], s["host_cu"][i + 1]
        if a == z:
            continue
        rows = s["cache"][s["table"][i, :-(-L // bs)].long()].reshape(-1, R + ROPE)[:L].float()
        keep = torch.arange(L, device=DEV) <= torch.arange(L - (z - a), L, device=DEV)[:, None]
        step = max(1, min(H, 2 ** 29 // max(1, (z - a) * L)))
        for h in range(0, H, step):
            wf = w[h:h + step].float()
            k = rows[:, :R] @ wf[:, :d].transpose(1, 2)
            v = rows[:, :R] @ wf[:, d:].transpose(1, 2)
            scores = qn[a:z, h:h + step].float().transpose(0, 1) @ k.transpose(1, 2)
            scores += qp[a:z, h:h + step].float().transpose(0, 1) @ rows[:, R:].T
            o = _softmax_times(scores * s["scale"], keep, v)
            out[a:z, h:h + step] = o.transpose(0, 1).to(out.dtype)
    return out


_plain = {"plan": _plain_plan, "append": _plain_append, "paged_decode": _plain_paged_decode,
          "latent_decode": _plain_latent_decode, "latent_prefill": _plain_latent_prefill}


# ------------------------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact[s["op"]](s)


def _exact_plan(s):
    """One request after another, one token after another."""
    table, free, bs = s["table"].tolist(), s["free"].tolist(), s["block"]
    cu, lens, slots, positions, taken = [0], [], [], [], 0
    for row, c, w in zip(table, s["ctx"].tolist(), s["new"].tolist()):
        for p in range(c, c + w):
            if p % bs == 0:
                row[p // bs] = free[taken]
                taken += 1
            slots.append(row[p // bs] * bs + p % bs)
            positions.append(p)
        cu.append(cu[-1] + w)
        lens.append(c + w)
    pad = s["tokens"] - len(slots)
    return [_ints(table), _ints(cu), _ints(lens),
            torch.tensor(slots + [-1] * pad, dtype=torch.int64, device=DEV),
            _ints(positions + [0] * pad), _ints([cu[-1], taken])]


def _exact_append(s):
    slots, bs = s["slots"], s["block"]
    if s["case"]["form"] == "latent":
        cache = s["cache_a"].double()
        R = s["a"].shape[1]
        flat = cache.view(-1, cache.shape[2])
        flat[:, :R].index_copy_(0, slots, s["a"].double())
        flat[:, R:].index_copy_(0, slots, s["b"].double())
        return [cache]
    out = []
    for rows, cache in ((s["a"], s["cache_a"]), (s["b"], s["cache_b"])):
        by_token = cache.double().transpose(1, 2).contiguous()
        by_token.view(-1, *by_token.shape[2:]).index_copy_(0, slots, rows.double())
        out.append(by_token.transpose(1, 2).contiguous())
    return out


def _exact_attend(q, k, v, first, scale):
    """q [h, t, d], k [h, L, d], v [h, L, e]; row i sees keys 0 .. first + i."""
    x = torch.matmul(k, q.transpose(1, 2)).mul_(scale)          # [h, L, t]
    seen = first + torch.arange(q.shape[1], device=DEV)
    x.masked_fill_(torch.arange(k.shape[1], device=DEV)[:, None] > seen[None, :], -math.inf)
    p = torch.softmax(x, dim=1).nan_to_num_(0.0)  # a row without keys gives zeros
    return torch.matmul(p.transpose(1, 2), v)


def _exact_paged_decode(s):
    q, bs = s["q"].double(), s["block"]
    n, P, H, d = q.shape
    kv = s["k_cache"].shape[1]
    out = torch.zeros_like(q)
    for i, L in enumerate(s["host_lens"]):
        ids = s["table"][i, :-(-L // bs)].long()
        for g in range(kv):
            k = s["k_cache"][ids, g].reshape(-1, d)[:L].double()
            v = s["v_cache"][ids, g].reshape(-1, d)[:L].double()
            h = slice(g * (H // kv), (g + 1) * (H // kv))
            o = _exact_attend(q[i, :, h].transpose(0, 1), k[None], v[None], L - P, s["scale"])
            out[i, :, h] = o.transpose(0, 1)
    return out


def _exact_latent(s, q_nope, q_pe, L, i, heads):
    """Keys and values written out for each head (q_* are [t, H, .])."""
    R, d, bs = s["w_kv"].shape[2], q_nope.shape[2], s["block"]
    rows = s["cache"][s["table"][i, :-(-L // bs)].long()].reshape(-1, R + ROPE)[:L].double()
    out = torch.empty_like(q_nope)
    for h in range(0, q_nope.shape[1], heads):
        w = s["w_kv"][h:h + heads].double()
        kv = torch.matmul(rows[:, :R], w.transpose(1, 2))       # [h, L, 2 d]
        k = torch.cat([kv[..., :d], rows[:, R:].expand(kv.shape[0], -1, -1)], dim=2)
        q = torch.cat([q_nope[:, h:h + heads], q_pe[:, h:h + heads]], dim=2).transpose(0, 1)
        o = _exact_attend(q, k, kv[..., d:].contiguous(), L - q.shape[1], s["scale"])
        out[:, h:h + heads] = o.transpose(0, 1)
    return out


def _exact_latent_decode(s):
    qn, qp = s["q_nope"].double(), s["q_pe"].double()
    return torch.stack([_exact_latent(s, qn[i], qp[i], L, i, 32)
                        for i, L in enumerate(s["host_lens"])])


def _exact_latent_prefill(s):
    qn, qp, cu = s["q_nope"].double(), s["q_pe"].double(), s["host_cu"]
    return torch.cat([_exact_latent(s, qn[cu[i]:cu[i + 1]], qp[cu[i]:cu[i + 1]], L, i, 4)
                      for i, L in enumerate(s["host_lens"])])


_exact = {"plan": _exact_plan, "append": _exact_append, "paged_decode": _exact_paged_decode,
          "latent_decode": _exact_latent_decode, "latent_prefill": _exact_latent_prefill}
