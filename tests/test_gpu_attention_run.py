"""The paged attention entry points as a serving loop uses them: a step's bookkeeping, append,
prefill and decode together and beside the gated delta-rule calls; captured graphs, other
streams, used workspaces, wide tables, large pools; rising scores; refusals on the GPU."""
import numpy as np
import pytest
import torch

import test_gpu_latent as lat
import test_gpu_paged as pag
from attn_util import assert_within, gen, normal, pages, tolerance
from gated_delta_rule_prefill_amd import gdn, inputs
from gpu_util import DEV, say
from oracle import attention
from test_gpu_debug_checks import debug_lib, expect_rejected

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ROPE = 64


def ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


# ------------------------------------------------------------------------- a whole run
def test_hybrid_model_run_matches_reference():
    """Chunked prompts, then decode steps, of a latent and a grouped-query layer over one set of
    block tables; the delta-rule layer of the same step takes the plan's cu_seqlens."""
    say("case run: plan, append, prefill, decode")
    g = gen(40)
    block, H, R, d, kv = 16, 4, 256, 64, 2
    prompts, n = [70, 5, 33, 128], 4
    n_blocks, width = 60, 12
    w = lat._weights(g, H, R, d)
    scale = (d + ROPE) ** -0.5
    cache = torch.full((n_blocks, block, R + ROPE), float("nan"), dtype=BF16, device=DEV)
    kc = torch.full((n_blocks, kv, block, d), float("nan"), dtype=BF16, device=DEV)
    vc = kc.clone()
    table = torch.full((n, width), -1, dtype=I32, device=DEV)
    free = torch.randperm(n_blocks, generator=g).to(I32).to(DEV)
    ctx, used = [0] * n, 0
    rows = [torch.empty(0, R + ROPE, dtype=BF16) for _ in range(n)]   # what the cache holds
    keys = [torch.empty(0, 2, kv, d, dtype=BF16) for _ in range(n)]
    steps = [[40, 5, 0, 64], [30, 0, 33, 64]] + [[1, 1, 1, 1]] * 3
    for step, new in enumerate(steps):
        T = sum(new)
        cu, lens, slots, pos, counts = gdn.gdn_paged_plan(ints(ctx), ints(new), table, free[used:],
                                                          block, T + 3)
        c, pe = normal(g, T + 3, R), normal(g, T + 3, ROPE)
        qkv = normal(g, T + 3, H + 2 * kv, d)     # a fused projection: q, k and v are its parts
        on = [x.to(DEV) for x in (c, pe, qkv)]
        gdn.gdn_latent_append(on[0], on[1], slots, cache)
        gdn.gdn_paged_append(on[2][:, H:H + kv], on[2][:, H + kv:], slots, kc, vc)
        at = 0
        for i, x in enumerate(new):
            rows[i] = torch.cat([rows[i], torch.cat([c, pe], 1)[at:at + x]])
            keys[i] = torch.cat([keys[i], qkv[at:at + x, H:].view(x, 2, kv, d)])
            at += x
        ctx = [a + b for a, b in zip(ctx, new)]
        used += int(counts[1])
        assert cu.tolist() == [0] + np.cumsum(new).tolist() and lens.tolist() == ctx
        assert pos[:T].tolist() == [p for i in range(n) for p in range(ctx[i] - new[i], ctx[i])]
        qn, qp = normal(g, T, H, d), normal(g, T, H, ROPE)
        limits = [(i, ctx[i] - new[i] + t + 1) for i in range(n) for t in range(new[i])]
        # the reference's own cache: request i's tokens in page i
        flat = torch.zeros(n, max(ctx), R + ROPE, dtype=BF16)
        for i in range(n):
            flat[i, :ctx[i]] = rows[i]
        own = torch.arange(n, dtype=I32).view(n, 1)
        want = attention.latent_expanded(qn, qp, w, flat.double(), own,
                                         [0] + np.cumsum(new).tolist(), ctx, scale)
        if step < 2:
            o = gdn.gdn_latent_prefill(qn.to(DEV), qp.to(DEV), w.to(DEV), cache, table, cu, lens,
                                       sum(ctx), scale=scale)
        else:
            o = gdn.gdn_latent_decode(qn.to(DEV), qp.to(DEV), w.to(DEV), cache, table, lens,
                                      scale=scale)
        tol = lat._tolerance(qn, qp, w, flat, own, limits, want, scale)
        assert_within(o, want, tol, f"latent, step {step}")
        if step >= 2:
            q = qkv[:T, :H].view(n, 1, H, d).contiguous()
            o = gdn.gdn_paged_decode(q.to(DEV), kc, vc, table, lens, scale=d ** -0.5)
            ref = torch.zeros(2, n, kv, max(ctx), d, dtype=BF16)
            for i in range(n):
                ref[:, i, :, :ctx[i]] = keys[i].permute(1, 2, 0, 3)
            want, mag, top = attention.paged_decode(q, ref[0].double(), ref[1].double(), own, ctx,
                                                    d ** -0.5)
            assert_within(o, want, tolerance(want, mag, top, d, max(ctx), BF16), f"step {step}")
        else:
            x = inputs.random_prefill(60 + step, new, H=2, dk=64, dv=64, chunk=64)
            args = [t.to(DEV) for t in (x.q, x.k, x.v, x.g, x.beta)]
            pools = [torch.zeros(n, 2, 64, 64, device=DEV) for _ in range(2)]
            slot = torch.arange(n, dtype=I32, device=DEV)
            a = gdn.gdn_prefill_chunked(*args, cu, 64, pools[0], slot, scale=x.scale)
            b = gdn.gdn_prefill_chunked(*args, x.cu_seqlens.to(DEV), 64, pools[1], slot,
                                        scale=x.scale)
            assert torch.equal(a, b) and torch.equal(*pools)


def test_requests_that_share_pages_and_repeat():
    """A prefix's pages in several block tables, one request listed twice."""
    say("case run: shared prefix")
    lens = [200, 90, 200, 131]
    case = list(pag._decode_case(41, lens, 1, 8, 2, 128, 16, BF16, poison=False))
    case[3][1, :4] = case[3][0, :4]
    case[3][2] = case[3][0]
    case[3][3, :4] = case[3][0, :4]
    case[0][2] = case[0][0]
    pag._check_decode(tuple(case))
    case = list(lat._decode_case(42, lens, 1, 4, 256, 64, 16, poison=False))
    case[4][1, :4] = case[4][0, :4]
    case[4][2] = case[4][0]
    lat._check_decode(tuple(case))


def test_more_requests_than_workgroups():
    say("case run: many short requests")
    lens = torch.randint(0, 40, (400,), generator=gen(43)).tolist()
    lens[5], lens[399] = 700, 0
    lat._check_decode(lat._decode_case(44, lens, 1, 2, 256, 64, 16))
    pag._check_decode(pag._decode_case(45, lens, 1, 4, 4, 64, 16, BF16))
    pag._check_decode(pag._decode_case(46, [0] * 9, 1, 4, 4, 64, 16, BF16))
    lat._check_decode(lat._decode_case(47, [0] * 9, 1, 4, 256, 64, 16))


# ----------------------------------------------------------------------- rising scores
def _ramp(n, kind):
    j = torch.arange(n)
    if kind == "rising":
        return j
    if kind == "falling":
        return n - 1 - j
    if kind == "steps":          # a new maximum every 50 keys, far above the last
        return j // 50 * 90
    return (j == n * 2 // 3) * 900 + (j == n - 1) * 800 - (j < 40) * 700  # spikes


def _parts(x):
    """x as a sum of two numbers that bf16 holds exactly (|x| < 2^16, whole)."""
    low = torch.remainder(x, 256)
    return low.to(BF16), (x - low).to(BF16)


@pytest.mark.parametrize("kind", ["rising", "falling", "steps", "spikes"])
@pytest.mark.parametrize("scale", [0.37, -0.37, 3.1, 0.0])
def test_scores_that_outgrow_the_reference(kind, scale):
    """Running maxima that rise by a little, by much, never, or are far below zero at first: the
    rescaling of sums and outputs. Scores are exact multiples of the scale."""
    say(f"case scores {kind} scale={scale}")
    n = 700
    low, high = _parts(_ramp(n, kind))
    case = list(pag._decode_case(50, [n, 330], 2, 8, 2, 64, 16, BF16, poison=False))
    q, kc, vc, table = case[:4]
    kc.zero_()
    j = torch.arange(n)
    page = table[0][j // 16].long()
    kc[page, :, j % 16, 0], kc[page, :, j % 16, 9] = low[:, None], high[:, None]
    j = torch.arange(330)
    page = table[1][j // 16].long()
    kc[page, :, j % 16, 0], kc[page, :, j % 16, 9] = low[:330, None], high[:330, None]
    q.zero_()
    q[..., 0], q[..., 9] = 1.0, 1.0
    case[5] = scale
    pag._check_decode(tuple(case))

    case = list(lat._decode_case(51, [n, 330], 2, 20, 256, 64, 16, poison=False))
    qn, qp, w, cache, table = case[:5]
    cache[..., 256:] = 0.0
    for i, m in ((0, n), (1, 330)):
        j = torch.arange(m)
        page = table[i][j // 16].long()
        cache[page, j % 16, 256], cache[page, j % 16, 261] = low[:m], high[:m]
    qn.zero_()
    qp.zero_()
    qp[..., 0], qp[..., 5] = 1.0, 1.0
    case[6] = scale
    lat._check_decode(tuple(case))

    T = 300                                    # of request 0's tokens, and all of request 1's
    case = [torch.zeros(T + 330, 2, 64, dtype=BF16), torch.zeros(T + 330, 2, ROPE, dtype=BF16),
            w[:2], cache, table, torch.tensor([0, T, T + 330], dtype=I32),
            torch.tensor([n, 330], dtype=I32), scale]
    case[1][..., 0], case[1][..., 5] = 1.0, 1.0
    lat._check_prefill(tuple(case), every=7)


@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_negative_and_zero_scales(scale):
    say(f"case scale {scale}")
    case = list(lat._decode_case(52, [130, 3, 0, 64], 2, 6, 512, 128, 16, q_scale=0.7))
    case[6] = scale
    lat._check_decode(tuple(case))
    case = list(lat._prefill_case(53, [0, 70], [130, 40], 2, 512, 128, 16, q_scale=0.7))
    case[7] = scale
    lat._check_prefill(tuple(case), every=3)


def test_nan_of_one_request_stays_with_it():
    """A NaN query row spoils itself only; NaN and infinite cache rows their own request."""
    say("case NaN kept apart")
    nan, lens = float("nan"), [200, 90, 300]
    for mod, q_at, rows in ((pag, 0, (1, 2)), (lat, 0, (3,))):
        if mod is pag:
            case = list(pag._decode_case(54, lens, 2, 8, 2, 64, 16, BF16, poison=False))
        else:
            case = list(lat._decode_case(55, lens, 2, 4, 256, 64, 16, poison=False))
        table = case[3] if mod is pag else case[4]
        want = mod._run_decode(tuple(case))
        bad = list(case)
        bad[q_at] = case[q_at].clone()
        bad[q_at][1, 0, 1, 3] = nan
        got = mod._run_decode(tuple(bad))
        assert torch.isnan(got[1, 0, 1].float()).all()
        mask = torch.ones(got.shape[:3], dtype=torch.bool)
        mask[1, 0, 1] = False
        assert torch.equal(got[mask], want[mask])
        bad = list(case)
        for r in rows:
            bad[r] = case[r].clone()
            bad[r][int(table[1, 2])] = nan if r % 2 else float("inf")
        got = mod._run_decode(tuple(bad))
        assert torch.isnan(got[1].float()).all()
        assert torch.equal(got[[0, 2]], want[[0, 2]])
    case = list(lat._prefill_case(56, [0, 30, 0], [70, 60, 130], 2, 256, 64, 16, poison=False))
    want = lat._run_prefill(tuple(case))
    bad = list(case)
    bad[0] = case[0].clone()
    bad[0][75, 1, 0] = nan
    got = lat._run_prefill(tuple(bad))
    assert torch.isnan(got[75, 1].float()).all()
    mask = torch.ones(got.shape[:2], dtype=torch.bool)
    mask[75, 1] = False
    assert torch.equal(got[mask], want[mask])
    bad = list(case)
    bad[3] = case[3].clone()
    bad[3][int(case[4][1, 0])] = nan
    got = lat._run_prefill(tuple(bad))
    assert torch.isnan(got[70:130].float()).all()
    assert torch.equal(got[:70], want[:70]) and torch.equal(got[130:], want[130:])


# ------------------------------------------------------------------ graphs and streams
class Step:
    """One decode step and one prompt of the whole set over static buffers."""

    def __init__(self, seed, lens=(500, 40, 0, 90)):
        g = gen(seed)
        self.g, self.block, self.H, self.n = g, 16, 8, len(lens)
        n, H, R, d, kv = self.n, 8, 256, 64, 2
        self.lens = list(lens)
        table, self.n_blocks = pages(g, [x + 40 for x in lens], 16)
        held = torch.tensor([-(-x // 16) for x in lens])
        self.free = table[torch.arange(table.shape[1])[None] >= held[:, None]]
        self.free = self.free[self.free >= 0].to(DEV)
        table[torch.arange(table.shape[1])[None] >= held[:, None]] = -1
        self.table0 = table.to(DEV)
        self.cache0 = normal(g, self.n_blocks, 16, R + ROPE).to(DEV)
        self.kc0, self.vc0 = (normal(g, self.n_blocks, kv, 16, d).to(DEV) for _ in range(2))
        self.w = lat._weights(g, H, R, d).to(DEV)
        self.ctx, self.new = ints(self.lens), ints([1] * n)
        self.T = 48
        self.rows = [torch.empty(self.T, x, dtype=BF16, device=DEV) for x in (R, ROPE)]
        self.kv = torch.empty(self.T, 2 * kv, d, dtype=BF16, device=DEV)
        self.q = torch.empty(n, H, d, dtype=BF16, device=DEV)
        self.qn = torch.empty(self.T, H, d, dtype=BF16, device=DEV)
        self.qp = torch.empty(self.T, H, ROPE, dtype=BF16, device=DEV)
        self.keys = 2000
        dims = (H, R, ROPE, d, d)
        self.sizes = (gdn.gdn_paged_decode_workspace_bytes(H, kv, d, BF16, n),
                      gdn.gdn_latent_decode_workspace_bytes(*dims, n),
                      gdn.gdn_latent_prefill_workspace_bytes(*dims, n, self.T, self.keys))
        self.ws = [torch.empty(s, dtype=torch.uint8, device=DEV) for s in self.sizes]
        self.reset()

    def reset(self):
        self.table, self.cache = self.table0.clone(), self.cache0.clone()
        self.kc, self.vc = self.kc0.clone(), self.vc0.clone()

    def fill(self, new):
        """The next step's inputs, into the static buffers."""
        self.new.copy_(torch.tensor(new, dtype=I32))
        for t in (*self.rows, self.kv, self.q, self.qn, self.qp):
            t.copy_(normal(self.g, *t.shape))

    def run(self, ws=None, stream=None):
        ws = self.ws if ws is None else ws
        cu, lens, slots, pos, counts = gdn.gdn_paged_plan(
            self.ctx, self.new, self.table, self.free, 16, self.T, stream=stream)
        gdn.gdn_latent_append(*self.rows, slots, self.cache, stream=stream)
        gdn.gdn_paged_append(self.kv[:, :2], self.kv[:, 2:], slots, self.kc, self.vc,
                             stream=stream)
        a = gdn.gdn_paged_decode(self.q, self.kc, self.vc, self.table, lens, scale=0.125,
                                 workspace=ws[0], stream=stream)
        b = gdn.gdn_latent_decode(self.qn[:self.n], self.qp[:self.n], self.w, self.cache,
                                  self.table, lens, scale=0.1, workspace=ws[1], stream=stream)
        c = torch.zeros_like(self.qn) if stream is None else None
        c = gdn.gdn_latent_prefill(self.qn, self.qp, self.w, self.cache, self.table, cu, lens,
                                   self.keys, scale=0.1, o=c, workspace=ws[2], stream=stream)
        return a, b, c, self.table, self.cache, slots, counts


NEW = [[1, 1, 1, 1], [7, 0, 30, 2], [0, 0, 0, 0], [16, 16, 1, 1]]


def test_graph_replays_match_eager():
    say("case graph: plan, append, decode, prefill")
    s = Step(70)
    s.fill(NEW[0])
    s.run()
    s.reset()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = s.run()
    table, cache, kc, vc = s.table, s.cache, s.kc, s.vc
    for new in NEW * 2:
        s.fill(new)
        s.reset()                                  # eager, on copies
        want = [t.clone() for t in s.run()]
        torch.cuda.synchronize()
        for dst, src in ((table, s.table0), (cache, s.cache0), (kc, s.kc0), (vc, s.vc0)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y), new


def test_two_graphs_with_a_workspace_each():
    say("case graph: two, replayed side by side")
    a, b = Step(71), Step(72, (33, 900))
    for s in (a, b):
        s.fill(NEW[0][:s.n])
        s.run()
        s.reset()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run())
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(3):
        want = []
        for s, out in zip((a, b), outs):
            s.fill([2, 5, 1, 1][:s.n])
            held = s.table, s.cache, s.kc, s.vc
            s.reset()
            want.append([t.clone() for t in s.run()])
            s.table, s.cache, s.kc, s.vc = held
            for dst, src in zip(held, (s.table0, s.cache0, s.kc0, s.vc0)):
                dst.copy_(src)
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for out, ref in zip(outs, want):
            for x, y in zip(out, ref):
                assert torch.equal(x, y)


@pytest.mark.parametrize("as_int", [False, True])
def test_on_another_stream(as_int):
    say(f"case stream as_int={as_int}")
    s = Step(73)
    s.fill(NEW[1])
    want = [t.clone() for t in s.run()]
    s.reset()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = s.run(ws=(None, None, None), stream=side.cuda_stream if as_int else side)
    side.synchronize()
    T = sum(NEW[1])
    for i, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x[:T], y[:T]) if i == 2 else torch.equal(x, y)


def test_workspaces_hold_anything_before():
    say("case dirty workspaces")
    s = Step(74)
    s.fill(NEW[1])
    want = [t.clone() for t in s.run()]
    for fill in (0xff, 0x00, 0x7f):
        s.reset()
        ws = [torch.full((x,), fill, dtype=torch.uint8, device=DEV) for x in s.sizes]
        for x, y in zip(s.run(ws), want):
            assert torch.equal(x, y), fill
    # one request after another in the same space: long, then short, then none
    big = [lat._decode_case(75, x, 1, 40, 256, 64, 16) for x in ([3000, 70], [5, 6], [0, 0])]
    ws = torch.full((gdn.gdn_latent_decode_workspace_bytes(40, 256, ROPE, 64, 64, 2),), 0xff,
                    dtype=torch.uint8, device=DEV)
    for case in big:
        assert torch.equal(lat._run_decode(case, workspace=ws), lat._run_decode(case))


# ------------------------------------------------------------------- tables and pools
def test_wide_tables_with_anything_behind_the_last_page():
    say("case wide tables")
    case = list(pag._decode_case(80, [100, 7, 0], 1, 8, 2, 64, 16, BF16))
    want = pag._run_decode(tuple(case))
    junk = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, 9000), generator=gen(81)).to(I32)
    narrow = case[3]
    for i, x in enumerate((7, 1, 0)):
        junk[i, :x] = narrow[i, :x]
    case[3] = junk
    assert torch.equal(pag._run_decode(tuple(case)), want)
    case = list(lat._prefill_case(82, [60, 0], [40, 7], 2, 256, 64, 16))
    want = lat._run_prefill(tuple(case))
    junk = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, 9000), generator=gen(83)).to(I32)
    for i, x in enumerate((7, 1)):
        junk[i, :x] = case[4][i, :x]
    case[4] = junk
    assert torch.equal(lat._run_prefill(tuple(case)), want)


def test_pools_past_32_bit_offsets():
    """Pages behind 4 GiB (and 2^31 elements) of a pool: written and read as in a small pool."""
    say("case large pools")
    lens, block = [300, 41], 64
    table, small = pages(gen(84), lens, block)
    T = sum(lens)
    slots = torch.cat([table[i][torch.arange(n) // block].long() * block + torch.arange(n) % block
                       for i, n in enumerate(lens)]).to(DEV)
    g = gen(85)
    c, pe = normal(g, T, 512).to(DEV), normal(g, T, ROPE).to(DEV)
    k, v = normal(g, T, 8, 128).to(DEV), normal(g, T, 8, 128).to(DEV)
    q, qn, qp = (normal(g, 2, 16, x).to(DEV) for x in (128, 128, ROPE))
    w = lat._weights(g, 16, 512, 128).to(DEV)
    ln = ints(lens)
    outs = []
    for first, blocks in ((0, small), (62000, 62000 + small)):
        # 62000 pages are 4.57 GB of latent rows, and 8.1 GB of keys
        t = torch.where(table >= 0, table + first, table).to(DEV)
        at = slots + first * block
        cache = torch.empty(blocks, block, 512 + ROPE, dtype=BF16, device=DEV)
        kc = torch.empty(blocks, 8, block, 128, dtype=BF16, device=DEV)
        vc = torch.empty_like(kc)
        for x in (cache, kc, vc):
            x[first:].zero_()
        gdn.gdn_latent_append(c, pe, at, cache)
        gdn.gdn_paged_append(k, v, at, kc, vc)
        outs.append((gdn.gdn_paged_decode(q, kc, vc, t, ln, scale=0.1),
                     gdn.gdn_latent_decode(qn, qp, w, cache, t, ln, scale=0.1),
                     gdn.gdn_latent_prefill(qn, qp, w, cache, t, ints([0, 1, 2]), ln, T,
                                            scale=0.1),
                     cache[first:].clone(), kc[first:].clone(), vc[first:].clone()))
        torch.cuda.synchronize()
        del cache, kc, vc
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    assert outs[0][0].float().abs().max() > 0.01 and outs[0][3].float().abs().max() > 1


# -------------------------------------------------------------------- sizes at the limits
@pytest.mark.parametrize("H,kv,P", [(1024, 1, 1), (1024, 1024, 1), (512, 1, 16)])
def test_most_heads_paged(H, kv, P):
    say(f"case limits paged H={H} kv={kv} P={P}")
    pag._check_decode(pag._decode_case(95, [37, 0, 150], P, H, kv, 64, 16, BF16))


@pytest.mark.parametrize("H,P", [(1024, 1), (128, 16)])
def test_most_heads_latent(H, P):
    say(f"case limits latent H={H} P={P}")
    lat._check_decode(lat._decode_case(96, [70, 0, 18], P, H, 256, 64, 16))
    if P == 1:
        lat._check_prefill(lat._prefill_case(97, [30, 0], [2, 1], H, 256, 64, 16))


def test_pages_of_one_token():
    say("case limits: block size 1")
    pag._check_decode(pag._decode_case(98, [130, 1, 0, 64], 2, 8, 2, 128, 1, BF16))
    lat._check_decode(lat._decode_case(99, [130, 1, 0, 64], 2, 4, 512, 128, 1))
    lat._check_prefill(lat._prefill_case(100, [0, 70], [66, 3], 2, 256, 64, 1))


def test_prefill_without_keys_gives_zeros():
    """total_keys 0 (and lengths of 0 under a positive one): no query sees a token."""
    say("case limits: no keys")
    case = list(lat._prefill_case(101, [0], [40], 2, 256, 64, 16))
    o = torch.full((40, 2, 64), 7.0, dtype=BF16, device=DEV)
    assert not lat._run_prefill(tuple(case), keys=0, o=o).any()
    case[6] = torch.zeros(1, dtype=I32)
    assert not lat._run_prefill(tuple(case), keys=64, o=o.fill_(7.0)).any()


# ---------------------------------------------------------------------------- refusals
def test_debug_library_rejects_repeated_cache_slots():
    say("case debug build: an append with a repeated cache slot")
    k = normal(gen(90), 5, 2, 64).to(DEV)
    kc = torch.zeros(4, 2, 16, 64, dtype=BF16, device=DEV)
    vc = torch.zeros_like(kc)
    cache = torch.zeros(4, 16, 128, dtype=BF16, device=DEV)
    dup = torch.tensor([3, 60, -1, 3, 64], dtype=torch.int64, device=DEV)
    fine = torch.tensor([3, 60, -1, 64, -1], dtype=torch.int64, device=DEV)
    with debug_lib():
        expect_rejected(lambda: gdn.gdn_paged_append(k, k, dup, kc, vc), "append")
        expect_rejected(lambda: gdn.gdn_latent_append(k[:, 0].contiguous(), k[:, 1].contiguous(),
                                                      dup, cache), "latent append")
        torch.cuda.synchronize()
        assert not kc.any() and not vc.any() and not cache.any()
        gdn.gdn_paged_append(k, k, fine, kc, vc)
        torch.cuda.synchronize()
        assert torch.equal(kc[0, :, 3], k[0]) and torch.equal(vc[3, :, 12], k[1])


def test_binding_refuses_what_does_not_fit():
    say("case binding refusals")
    q, kc, vc, table, lens, _ = (x.to(DEV) if torch.is_tensor(x) else x for x in
                                 pag._decode_case(91, [20, 3], 1, 8, 2, 64, 16, BF16))
    call = gdn.gdn_paged_decode
    for bad in ((q.float(), kc, vc, table, lens), (q, kc.float(), vc, table, lens),
                (q, kc, vc[:-1], table, lens), (q, kc, vc, table.long(), lens),
                (q, kc, vc, table[:1], lens), (q, kc, vc, table[0], lens),
                (q, kc, vc, table, lens.long()), (q, kc, vc, table, lens[:1]),
                (q, kc.transpose(1, 2), vc, table, lens), (q, kc, vc, table[:, ::2], lens),
                (q.transpose(1, 2), kc, vc, table, lens), (q, kc, vc, table.cpu(), lens),
                (q, kc, vc.cpu(), table, lens)):
        with pytest.raises((ValueError, gdn.GdnError)):
            call(*bad)
    with pytest.raises(ValueError):
        call(q, kc, vc, table, lens, o=torch.empty_like(q)[..., :32])
    with pytest.raises(gdn.GdnError) as e:
        call(q, kc, vc, table, lens, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5
    with pytest.raises(gdn.GdnError) as e:     # 6 heads over 4
        call(q[:, :, :6].contiguous(), torch.cat([kc, kc], 1), torch.cat([vc, vc], 1), table, lens)
    assert e.value.status == 2
    slots = torch.zeros(3, dtype=torch.int64, device=DEV)
    k = torch.zeros(3, 2, 64, dtype=BF16, device=DEV)
    for bad in ((k, k, slots.int(), kc, vc), (k, k[:2], slots, kc, vc), (k, k, slots[:2], kc, vc),
                (k.transpose(0, 1), k, slots, kc, vc),
                (torch.zeros(3, 64, 2, dtype=BF16, device=DEV).transpose(1, 2), k, slots, kc, vc),
                (k, k.float(), slots, kc, vc), (k, k, slots, kc, vc.float())):
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.gdn_paged_append(*bad)
    qn, qp, w, cache, table, lens, _ = (x.to(DEV) if torch.is_tensor(x) else x for x in
                                        lat._decode_case(92, [20, 3], 1, 4, 256, 64, 16))
    for bad in ((qn, qp[..., :32], w, cache, table, lens), (qn, qp, w.float(), cache, table, lens),
                (qn, qp, w[:, :, :128], cache, table, lens), (qn, qp, w[:2], cache, table, lens),
                (qn, qp, w, cache[..., :256], table, lens),
                (qn, qp[:1], w, cache, table, lens), (qn.float(), qp, w, cache, table, lens)):
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.gdn_latent_decode(*bad)
    with pytest.raises(ValueError):
        gdn.gdn_latent_prefill(qn[:, 0], qp[:, 0], w, cache, table, ints([0, 2]), lens, 23)
    ok = gdn.gdn_latent_prefill(qn[:, 0].contiguous(), qp[:, 0].contiguous(), w, cache, table,
                                ints([0, 1, 2]), lens, 23)
    torch.cuda.synchronize()
    assert torch.isfinite(ok.float()).all()
