"""Shared pages, prompts and decode behind shared prefixes as a serving loop uses them: a whole run
with forks, ends and a compaction between the steps; captured graphs, other streams, used
workspaces, large pools; refusals on the GPU and the debug library's checks."""
import numpy as np
import pytest
import torch

import test_gpu_paged_prefill as pre
import test_gpu_shared_decode as sha
from attn_util import assert_within, gen, normal, tolerance
from gated_delta_rule_prefill_amd import gdn, inputs
from gpu_util import DEV, say
from oracle import pages as oracle_pages
from test_gpu_debug_checks import debug_lib

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def ints(x):
    return torch.tensor(np.asarray(x), dtype=I32, device=DEV)


class Engine:
    """What a serving program keeps: table, free list, lengths; and every request's rows, packed
    and in order, as the reference."""

    def __init__(self, rows, width, n_blocks, block, H, kv, d, dtype, seed):
        self.g = gen(seed)
        self.block, self.H, self.kv, self.d, self.dtype = block, H, kv, d, dtype
        self.table = torch.full((rows, width), -1, dtype=I32, device=DEV)
        self.shares = torch.zeros(n_blocks, dtype=I32, device=DEV)
        self.kc = torch.full((n_blocks, kv, block, d), float("nan"), dtype=dtype, device=DEV)
        self.vc = self.kc.clone()
        self.free = torch.randperm(n_blocks, generator=self.g).to(I32).to(DEV)
        self.lens = [0] * rows
        self.held = [torch.empty(0, 2, kv, d, dtype=dtype) for _ in range(rows)]
        self.scale = d ** -0.5

    def take(self, n):
        self.free = self.free[n:]

    def step(self, new, attend):
        """new[i] tokens for every row; attend(q, cu, seq_lens) -> outputs, checked."""
        T = sum(new)
        cu, lens, slots, _, counts = gdn.gdn_paged_plan(ints(self.lens), ints(new), self.table,
                                                        self.free, self.block, T + 2)
        qkv = normal(self.g, T + 2, self.H + 2 * self.kv, self.d, dtype=self.dtype)
        on, H, kv = qkv.to(DEV), self.H, self.kv
        gdn.gdn_paged_append(on[:, H:H + kv], on[:, H + kv:], slots, self.kc, self.vc)
        at = 0
        for i, w in enumerate(new):
            self.held[i] = torch.cat([self.held[i], qkv[at:at + w, H:].view(w, 2, kv, self.d)])
            self.lens[i] += w
            at += w
        self.take(int(counts[1]))
        q = on[:T, :H].contiguous()
        o = attend(q, cu, lens)
        want, mag, top = self.expected(q.cpu(), new)
        assert_within(o.reshape(T, H, self.d), want,
                      tolerance(want, mag, top, self.d, max(self.lens), self.dtype), "step")

    def expected(self, q, new):
        """The newest tokens over the rows that each request holds, page by page of their own."""
        n, b = max(self.lens), self.block
        width = -(-n // b)
        k = torch.zeros(len(self.lens) * width, self.kv, b, self.d)
        v = k.clone()
        for i, rows in enumerate(self.held):
            for c, x in ((k, rows[:, 0]), (v, rows[:, 1])):
                pad = torch.zeros(width * b, self.kv, self.d)
                pad[:len(x)] = x.float()
                c[i * width:(i + 1) * width] = pad.view(width, b, self.kv, self.d).transpose(1, 2)
        table = np.arange(len(self.lens) * width).reshape(-1, width)
        cu = np.concatenate([[0], np.cumsum(new)])
        return oracle_pages.prefill(q.float(), k, v, table, cu, self.lens, self.scale)

    def prefill(self, q, cu, lens):
        return gdn.gdn_paged_prefill(q, self.kc, self.vc, self.table, cu, lens, scale=self.scale)


@pytest.mark.parametrize("dtype,d,block", [(BF16, 128, 16), (F32, 64, 24)])
def test_a_serving_run(gpu_lib, dtype, d, block):
    """Two prompts, four samples of the first and two of the second forked at several lengths with
    the linear layer's state, decode and verify steps over groups, two samples ended, the pool
    compacted, a further turn and further steps."""
    say("run", dtype, d, block)
    rows, H, kv = 8, 8, 2
    e = Engine(rows, 40, 260, block, H, kv, d, dtype, 70)
    st = torch.randn(rows, 2, 32, 32, generator=e.g).to(DEV)     # state pool of a linear layer
    e.step([150, 0, 0, 0, 0, 70, 0, 0], e.prefill)
    # forks: the whole prompt three times, 100 tokens of it once; of the second, 70 and 33
    src, dst, n = [0, 0, 0, 0, 5, 5], [1, 2, 3, 4, 6, 7], [150, 150, 150, 100, 70, 33]
    a, b, counts = gdn.gdn_paged_fork(ints(src), ints(dst), ints(n), e.table, block, e.shares,
                                      e.free)
    gdn.gdn_paged_copy([e.kc, e.vc], a, b)
    gdn.gdn_paged_copy([st], ints(src), ints(dst))               # a slot is a page
    e.take(int(counts[1]))
    assert int(counts[0]) == int(counts[1]) == sum(x % block > 0 for x in n)
    for s, t, x in zip(src, dst, n):
        e.lens[t], e.held[t] = x, e.held[s][:x]
        assert torch.equal(st[s], st[t])
    whole = [100 // block * block, 33 // block * block]
    cu, prefix = ints([0, 5, 8]), ints(whole)

    def shared(P):
        def attend(q, _, lens):
            return gdn.gdn_paged_shared_decode(q.view(-1, P, H, d), e.kc, e.vc, e.table, lens, cu,
                                               prefix, scale=e.scale, min_bytes=0)
        return attend
    for P in (1, 1, 3, 1):
        e.step([P] * rows, shared(P))
    # samples 2 and 6 end; their places stay empty
    ends = [2, 6]
    freed, counts = gdn.gdn_paged_free(ints(ends), ints([e.lens[i] for i in ends]), e.table, block,
                                       e.shares)
    got = freed[:int(counts[0])]
    assert not set(got.cpu().tolist()) & set(e.table[e.table >= 0].cpu().tolist())
    e.free = torch.cat([e.free, got])
    for i in ends:
        e.lens[i], e.held[i] = 0, e.held[i][:0]
    a, b, counts = gdn.gdn_paged_compact(ints(e.lens), e.table, block, e.shares)
    gdn.gdn_paged_copy([e.kc, e.vc], a, b, count=counts[1:])
    live = int(counts[0])
    e.free = torch.arange(live, e.shares.numel(), dtype=I32, device=DEV)
    held = {int(p) for i, n in enumerate(e.lens) for p in e.table[i, :-(-n // block)].cpu()}
    assert held == set(range(live))
    assert int(e.shares.sum()) == sum(-(-n // block) for n in e.lens) - live
    # a turn of several tokens for some, then single tokens for all that run
    e.step([20, 1, 0, 45, 3, 0, 0, 7], e.prefill)
    running = [1, 1, 0, 1, 1, 1, 0, 1]
    e.step(running, e.prefill)
    q = normal(e.g, rows, H, d, dtype=dtype)
    o = gdn.gdn_paged_shared_decode(q.to(DEV), e.kc, e.vc, e.table, ints(e.lens), cu, prefix,
                                    scale=e.scale)
    want, mag, top = e.expected(q[[i for i in range(rows) if running[i]]], running)
    assert_within(o[[i for i in range(rows) if running[i]]], want,
                  tolerance(want, mag, top, d, max(e.lens), dtype), "padded batch")
    assert bool((o[2] == 0).all()) and bool((o[6] == 0).all())


def test_captured_graph_of_a_step(gpu_lib):
    """Fork, copy, prompt, shared decode, end and compaction recorded once and replayed, with other
    inputs in between, against eager calls on the same inputs."""
    H, kv, d, block = 8, 2, 64, 16
    args = [x.to(DEV) for x in sha.make(50, [3, 2], [200, 90], [30] * 6, 1, H, kv, d, block, BF16)]
    q, kc, vc, table, lens, cu, prefix = args
    pq, pk, pv, ptable, pcu, plens = [x.to(DEV) for x in pre.make(51, [90, 300], [40, 130], H, kv, d,
                                                                   block, BF16)]
    kc, vc = torch.nan_to_num(kc), torch.nan_to_num(vc)
    rows, pool = 6, kc.shape[0] + 40
    kc, vc = (torch.cat([c, torch.zeros(40, *c.shape[1:], dtype=BF16, device=DEV)]) for c in (kc, vc))
    free = torch.arange(pool - 40, pool, dtype=I32, device=DEV)
    big = torch.full((rows + 4, table.shape[1]), -1, dtype=I32, device=DEV)
    big[:rows] = table
    state = dict(table=big, shares=torch.zeros(pool, dtype=I32, device=DEV), kc=kc, vc=vc, q=q, pq=pq)
    src, dst, flen = ints([0, 4]), ints([rows, rows + 1]), ints([205, 95])
    all_lens = torch.cat([lens, ints([205, 95, 0, 0])])

    def call(s):
        a, b, n = gdn.gdn_paged_fork(src, dst, flen, s["table"], block, s["shares"], free)
        gdn.gdn_paged_copy([s["kc"], s["vc"]], a, b)
        o = gdn.gdn_paged_shared_decode(s["q"], s["kc"], s["vc"], s["table"][:rows], lens, cu, prefix,
                                        scale=0.125, min_bytes=0)
        p = gdn.gdn_paged_prefill(s["pq"], pk, pv, ptable, pcu, plens, scale=0.125)
        freed, k = gdn.gdn_paged_free(ints_1, flen[1:], s["table"], block, s["shares"])
        after = torch.where(torch.arange(rows + 4, device=DEV) == rows + 1, 0, all_lens).to(I32)
        x, y, m = gdn.gdn_paged_compact(after, s["table"], block, s["shares"])
        gdn.gdn_paged_copy([s["kc"], s["vc"]], x, y, count=m[1:])
        return [a, b, n, o, p, freed, k, x, y, m, s["table"], s["shares"], s["kc"], s["vc"]]

    ints_1 = ints([rows + 1])
    fixed = {k: v.clone() for k, v in state.items()}
    for _ in range(2):
        call({k: v.clone() for k, v in state.items()})
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(fixed)
    for turn in range(4):
        g = gen(90 + turn)
        now = {k: v.clone() for k, v in state.items()}
        now["q"] = normal(g, *q.shape).to(DEV)
        now["pq"] = normal(g, *pq.shape).to(DEV)
        for k in fixed:
            fixed[k].copy_(now[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        want = call(now)
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), f"replay {turn}: output {i}"


def test_other_streams_and_used_workspaces(gpu_lib):
    """Calls on a given stream, workspaces full of NaN, and calls that follow each other in one
    workspace give the default call's bits."""
    a = [x.to(DEV) for x in sha.make(60, [4], [300], [40] * 5, 2, 8, 2, 128, 16, BF16)]
    b = [x.to(DEV) for x in pre.make(61, [400, 90], [300, 1], 8, 2, 128, 16, BF16)]
    want = gdn.gdn_paged_shared_decode(*a, scale=0.1, min_bytes=0), gdn.gdn_paged_prefill(*b, scale=0.1)
    size = max(gdn.gdn_paged_shared_decode_workspace_bytes(8, 2, 128, BF16, 5, 2, 1),
               gdn.gdn_paged_prefill_workspace_bytes(8, 2, 128, BF16, 2, 301))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        for _ in range(2):
            x = gdn.gdn_paged_shared_decode(*a, scale=0.1, min_bytes=0, workspace=ws, stream=stream)
            y = gdn.gdn_paged_prefill(*b, scale=0.1, workspace=ws, stream=stream)
        z = gdn.gdn_paged_shared_decode(*a, scale=0.1, min_bytes=0, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(y, want[1]) and torch.equal(z, want[0])
    with torch.cuda.stream(side):
        x, y = gdn.gdn_paged_shared_decode(*a, scale=0.1, min_bytes=0), gdn.gdn_paged_prefill(*b, scale=0.1)
    torch.cuda.synchronize()
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_two_calls_at_once_with_a_workspace_each(gpu_lib):
    a = [x.to(DEV) for x in pre.make(62, [900], [700], 16, 4, 64, 16, BF16)]
    want = gdn.gdn_paged_prefill(*a, scale=0.1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(gdn.gdn_paged_prefill(*a, scale=0.1))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)


def test_pools_beyond_four_gigabytes(gpu_lib):
    """Pages at both ends of caches whose byte offsets pass 32 bits."""
    H, kv, d, block, n_blocks = 16, 8, 128, 64, 40000
    page = kv * block * d
    assert n_blocks * page * 2 > 2 ** 32
    kc = torch.empty(n_blocks, kv, block, d, dtype=BF16, device=DEV)
    vc = torch.empty_like(kc)
    g = gen(63)
    ids = [3, 39999, 36000, 5, 39998, 20011]
    small_k, small_v = normal(g, 6, kv, block, d), normal(g, 6, kv, block, d)
    for i, p in enumerate(ids[:4]):
        kc[p], vc[p] = small_k[i].to(DEV), small_v[i].to(DEV)
    gdn.gdn_paged_copy([kc, vc], ints([39999, 3]), ints([39998, 20011]))
    small_k[4:], small_v[4:] = small_k[[1, 0]], small_v[[1, 0]]
    assert torch.equal(kc[39998].cpu(), small_k[4]) and torch.equal(vc[20011].cpu(), small_v[5])
    table, near = ints([ids[:3], ids[3:]]), ints([[0, 1, 2], [3, 4, 5]])
    q, cu, lens = normal(g, 70, H, d).to(DEV), ints([0, 50, 70]), ints([192, 180])
    sk, sv = small_k.to(DEV), small_v.to(DEV)
    far = gdn.gdn_paged_prefill(q, kc, vc, table, cu, lens, scale=0.1)
    assert torch.equal(far, gdn.gdn_paged_prefill(q, sk, sv, near, cu, lens, scale=0.1))
    two = ints([[ids[1], ids[2], ids[0]], [ids[1], ids[2], ids[4]]])
    two_near = ints([[1, 2, 0], [1, 2, 4]])
    rest = q[:2].contiguous(), lens, ints([0, 2]), ints([128])
    for least in (0, 2 ** 62):
        far = gdn.gdn_paged_shared_decode(rest[0], kc, vc, two, *rest[1:], scale=0.1, min_bytes=least)
        near = gdn.gdn_paged_shared_decode(rest[0], sk, sv, two_near, *rest[1:], scale=0.1,
                                           min_bytes=least)
        assert torch.equal(far, near)


def test_states_fork_with_their_requests(gpu_lib):
    """A forked slot of a state pool decodes as the original one does."""
    H, d = 2, 64
    pool = inputs.decode_pool(64, 6, H, d, d).to(DEV)
    gdn.gdn_paged_copy([pool], ints([1, 1]), ints([4, 0]))
    st = inputs.DecodeStream(65, 1, H, d, d, dtype=BF16)
    q, k, v, g, b = (t.to(DEV).repeat(3, *[1] * (t.dim() - 1)) for t in st.next())
    o = gdn.gdn_decode_step(q, k, v, g, b, pool, ints([1, 4, 0]))
    assert torch.equal(o[0], o[1]) and torch.equal(o[0], o[2])
    assert torch.equal(pool[1], pool[4]) and torch.equal(pool[1], pool[0])


def test_binding_refusals(gpu_lib):
    q, k, v, table, cu, lens = (x.to(DEV) for x in pre.make(66, [40], [40], 4, 2, 64, 16, BF16))
    for bad in (dict(q=q[:, ::2]), dict(q=q.float()), dict(k=k[:, :1]), dict(v=v[:-1]),
                dict(table=table.long()), dict(table=table[0]), dict(cu=cu[:1]), dict(cu=cu.cpu()),
                dict(lens=lens.long())):
        a = {**dict(q=q, k=k, v=v, table=table, cu=cu, lens=lens), **bad}
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_paged_prefill(*a.values())
    with pytest.raises(gdn.GdnError):
        gdn.gdn_paged_prefill(q, k, v, table, cu, lens,
                              workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    one, t = ints([0]), ints([[1, 2]])
    shares = ints([0] * 8)
    for bad in (lambda: gdn.gdn_paged_fork(one, ints([1, 2]), one, t, 16, shares, one),
                lambda: gdn.gdn_paged_fork(one, one, one, ints([[1, 2], [3, 4]])[:, :1], 16, shares,
                                           one),
                lambda: gdn.gdn_paged_free(one.long(), one, t, 16, shares),
                lambda: gdn.gdn_paged_compact(ints([1, 2]), t, 16, shares),
                lambda: gdn.gdn_paged_shared_decode(q, k, v, table.repeat(40, 1), lens.repeat(40), one,
                                                    one)):
        with pytest.raises(ValueError):
            bad()


def test_debug_library_checks_pairs(gpu_lib):
    cache = torch.arange(80, dtype=F32, device=DEV).view(10, 8)
    keep = cache.clone()
    t, s, free = ints([[1, 2]] * 7), ints([0] * 10), ints([7, 8])
    with debug_lib():
        for a, b, what in (([0, 1], [5, 5], "used twice"), ([0, 5], [5, 6], "source")):
            with pytest.raises(gdn.GdnError, match=what):
                gdn.gdn_paged_copy([cache], ints(a), ints(b))
            with pytest.raises(gdn.GdnError, match=what):
                gdn.gdn_paged_fork(ints(a), ints(b), ints([20, 20]), t, 16, s, free)
        assert torch.equal(cache, keep) and t.cpu().tolist() == [[1, 2]] * 7
        # skipped pairs and those behind the count are not looked at
        gdn.gdn_paged_copy([cache], ints([-1, 0, 3]), ints([5, 5, 0]), count=ints([2]))
        assert torch.equal(cache[5], keep[0])
        gdn.gdn_paged_fork(ints([0, -1]), ints([5, 5]), ints([20, 20]), t, 16, s, free)
    assert t[5].cpu().tolist() == [1, 7]
