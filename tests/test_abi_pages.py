"""Refusals, sizes and no-ops of the entry points for shared pages, prompts and decode behind shared
prefixes, on a host without a GPU: bad arguments are turned down before any HIP call."""
import ctypes

import pytest

from gated_delta_rule_prefill_amd import gdn
from gated_delta_rule_prefill_amd.gdn import gdn_paged_dims_t

FAKE = 0x7f0000000000  # aligned, never dereferenced
NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4, 5
I32_MAX = 2 ** 31 - 1


def call(name, defaults, kw):
    unknown = set(kw) - set(defaults)
    assert not unknown, unknown
    return getattr(gdn.load(), name)(*{**defaults, **kw}.values())


def refused(status, got):
    assert got == status
    assert gdn.gdn_last_error() != ""


FORK = dict(src_rows=FAKE, dst_rows=FAKE, fork_lens=FAKE, n=3, block_table=FAKE, n_rows=9,
            max_blocks=8, block_size=16, shares=FAKE, n_blocks=50, free_blocks=FAKE, n_free=5,
            copy_src=FAKE, copy_dst=FAKE, counts=FAKE, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(src_rows=None), NULL), (dict(dst_rows=None), NULL), (dict(fork_lens=None), NULL),
    (dict(block_table=None), NULL), (dict(shares=None), NULL), (dict(free_blocks=None), NULL),
    (dict(copy_src=None), NULL), (dict(copy_dst=None), NULL), (dict(counts=None), NULL),
    (dict(n=0, counts=None), NULL),
    (dict(src_rows=FAKE + 2), ALIGN), (dict(block_table=FAKE + 4), ALIGN),
    (dict(shares=FAKE + 8), ALIGN), (dict(counts=FAKE + 1), ALIGN), (dict(copy_dst=FAKE + 3), ALIGN),
    (dict(n=-1), SHAPE), (dict(n_rows=-1), SHAPE), (dict(n_blocks=0), SHAPE),
    (dict(block_size=0), SHAPE), (dict(max_blocks=0), SHAPE), (dict(n_free=-1), SHAPE),
    (dict(n=(1 << 24) + 1), UNSUPPORTED), (dict(n_rows=(1 << 24) + 1), UNSUPPORTED),
    (dict(max_blocks=1 << 26), UNSUPPORTED),
])
def test_fork_refuses(kw, status):
    refused(status, call("gdn_paged_fork", FORK, kw))


FREE = dict(rows=FAKE, lens=FAKE, n=3, block_table=FAKE, n_rows=9, max_blocks=8, block_size=16,
            shares=FAKE, n_blocks=50, freed=FAKE, max_freed=24, counts=FAKE, workspace=FAKE,
            ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=None), NULL), (dict(lens=None), NULL), (dict(block_table=None), NULL),
    (dict(shares=None), NULL), (dict(freed=None), NULL), (dict(counts=None), NULL),
    (dict(workspace=None), NULL),
    (dict(freed=FAKE + 2), ALIGN), (dict(shares=FAKE + 4), ALIGN), (dict(workspace=FAKE + 8), ALIGN),
    (dict(n=-1), SHAPE), (dict(max_freed=-1), SHAPE), (dict(n_blocks=-5), SHAPE),
    (dict(block_size=-1), SHAPE), (dict(max_blocks=-1), SHAPE),
    (dict(max_blocks=I32_MAX), UNSUPPORTED), (dict(n=I32_MAX), UNSUPPORTED),
    (dict(ws_bytes=0), WORKSPACE), (dict(n_blocks=1 << 20, ws_bytes=1000), WORKSPACE),
])
def test_free_refuses(kw, status):
    refused(status, call("gdn_paged_free", FREE, kw))


COMPACT = dict(seq_lens=FAKE, n_rows=9, block_table=FAKE, max_blocks=8, block_size=16, shares=FAKE,
               n_blocks=50, copy_src=FAKE, copy_dst=FAKE, max_copies=25, counts=FAKE,
               workspace=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(seq_lens=None), NULL), (dict(block_table=None), NULL), (dict(shares=None), NULL),
    (dict(copy_src=None), NULL), (dict(copy_dst=None), NULL), (dict(counts=None), NULL),
    (dict(workspace=None), NULL),
    (dict(seq_lens=FAKE + 1), ALIGN), (dict(block_table=FAKE + 8), ALIGN),
    (dict(copy_src=FAKE + 2), ALIGN), (dict(workspace=FAKE + 4), ALIGN),
    (dict(n_rows=-1), SHAPE), (dict(max_copies=-1), SHAPE), (dict(n_blocks=0), SHAPE),
    (dict(block_size=0), SHAPE), (dict(max_blocks=0), SHAPE),
    (dict(n_rows=1 << 25), UNSUPPORTED), (dict(ws_bytes=15), WORKSPACE),
])
def test_compact_refuses(kw, status):
    refused(status, call("gdn_paged_compact", COMPACT, kw))


def pools(*addresses):
    return (ctypes.c_void_p * len(addresses))(*addresses)


COPY = dict(caches=pools(FAKE, FAKE + 4096), n_caches=2, page_bytes=1024, n_blocks=50,
            copy_src=FAKE, copy_dst=FAKE, n=4, count=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(caches=None), NULL), (dict(caches=pools(FAKE, None)), NULL), (dict(copy_src=None), NULL),
    (dict(copy_dst=None), NULL),
    (dict(caches=pools(FAKE, FAKE + 8)), ALIGN), (dict(copy_src=FAKE + 2), ALIGN),
    (dict(count=FAKE + 1), ALIGN),
    (dict(n_caches=-1), SHAPE), (dict(n=-1), SHAPE), (dict(n_blocks=0), SHAPE),
    (dict(page_bytes=0), SHAPE), (dict(page_bytes=-16), SHAPE),
    (dict(n_caches=129), UNSUPPORTED), (dict(page_bytes=1000), UNSUPPORTED),
    (dict(page_bytes=1 << 41), UNSUPPORTED),
])
def test_copy_refuses(kw, status):
    refused(status, call("gdn_paged_copy", COPY, kw))


def paged(H=32, kv=8, d=128, dtype=1):
    return ctypes.byref(gdn_paged_dims_t(H, kv, d, dtype, 0.1))


SHARED = dict(dims=paged(), q=FAKE, k_cache=FAKE, v_cache=FAKE, n_blocks=100, block_size=16,
              block_table=FAKE, max_blocks=20, seq_lens=FAKE, batch=6, n_pos=1, group_cu=FAKE,
              prefix_lens=FAKE, n_groups=2, min_bytes=-1, o=FAKE, workspace=FAKE, ws_bytes=1 << 40, stream=None)
PREFILL = dict(dims=paged(), q=FAKE, k_cache=FAKE, v_cache=FAKE, n_blocks=100, block_size=16,
               block_table=FAKE, max_blocks=20, cu_seqlens=FAKE, seq_lens=FAKE, n_seqs=3,
               total_tokens=50, o=FAKE, workspace=FAKE, ws_bytes=1 << 40, stream=None)
BOTH = [
    (dict(dims=None), NULL), (dict(q=None), NULL), (dict(k_cache=None), NULL),
    (dict(v_cache=None), NULL), (dict(block_table=None), NULL), (dict(seq_lens=None), NULL),
    (dict(o=None), NULL), (dict(workspace=None), NULL),
    (dict(q=FAKE + 8), ALIGN), (dict(v_cache=FAKE + 8), ALIGN), (dict(workspace=FAKE + 8), ALIGN),
    (dict(block_table=FAKE + 4), ALIGN), (dict(seq_lens=FAKE + 4), ALIGN),
    (dict(dims=paged(H=0)), SHAPE), (dict(dims=paged(kv=0)), SHAPE), (dict(dims=paged(H=30)), SHAPE),
    (dict(n_blocks=0), SHAPE), (dict(block_size=0), SHAPE), (dict(max_blocks=0), SHAPE),
    (dict(dims=paged(H=1032)), UNSUPPORTED), (dict(dims=paged(d=96)), UNSUPPORTED),
    (dict(dims=paged(dtype=2)), UNSUPPORTED), (dict(max_blocks=1 << 26), UNSUPPORTED),
    (dict(n_blocks=1 << 28), UNSUPPORTED), (dict(ws_bytes=1000), WORKSPACE),
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(group_cu=None), NULL), (dict(prefix_lens=None), NULL), (dict(group_cu=FAKE + 2), ALIGN),
    (dict(batch=-1), SHAPE), (dict(n_groups=-1), SHAPE), (dict(n_pos=0), UNSUPPORTED),
    (dict(n_pos=17), UNSUPPORTED), (dict(max_blocks=1 << 22, batch=1 << 8), UNSUPPORTED),
    (dict(batch=1 << 23, n_pos=16, max_blocks=1), UNSUPPORTED), (dict(n_groups=1 << 25), UNSUPPORTED),
    (dict(dims=paged(H=8), batch=1 << 21, max_blocks=1), UNSUPPORTED),
])
def test_shared_decode_refuses(kw, status):
    refused(status, call("gdn_paged_shared_decode", SHARED, kw))


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(cu_seqlens=None), NULL), (dict(cu_seqlens=FAKE + 4), ALIGN), (dict(n_seqs=-1), SHAPE),
    (dict(total_tokens=-1), SHAPE), (dict(total_tokens=1 << 27), UNSUPPORTED),
    (dict(n_seqs=1 << 25), UNSUPPORTED),
])
def test_prefill_refuses(kw, status):
    refused(status, call("gdn_paged_prefill", PREFILL, kw))


def test_workspaces_are_exact():
    lib = gdn.load()
    for name, defaults, need in [
        ("gdn_paged_free", FREE, gdn.gdn_paged_free_workspace_bytes(50)),
        ("gdn_paged_compact", COMPACT, gdn.gdn_paged_compact_workspace_bytes(50)),
        ("gdn_paged_shared_decode", SHARED,
         gdn.gdn_paged_shared_decode_workspace_bytes(32, 8, 128, 1, 6, 1, 2)),
        ("gdn_paged_prefill", PREFILL, gdn.gdn_paged_prefill_workspace_bytes(32, 8, 128, 1, 3, 50)),
    ]:
        assert call(name, defaults, dict(ws_bytes=need - 1)) == WORKSPACE, name
        assert need > 0
    assert lib.gdn_paged_free_workspace_bytes(50, None) == NULL
    assert lib.gdn_paged_compact_workspace_bytes(0, ctypes.byref(ctypes.c_size_t())) == SHAPE
    assert lib.gdn_paged_prefill_workspace_bytes(paged(), 1, 1, None) == NULL
    # a bit and a count for every 32 pages
    assert gdn.gdn_paged_compact_workspace_bytes(1 << 20) == 2 * (1 << 20) // 8
    # no parts beyond those of the workers, whatever the lengths: 32 bytes and a position a tile
    one, many = (gdn.gdn_paged_prefill_workspace_bytes(32, 8, 128, 1, 1, t) for t in (64, 64 << 12))
    assert 0 < many - one < (64 << 12) * 4 / 256 * 40 + 4096
    # groups beyond half the batch have nothing to share
    args = (32, 8, 128, 1, 40, 2)
    sizes = [gdn.gdn_paged_shared_decode_workspace_bytes(*args, n) for n in (20, 40, 400)]
    assert sizes[2] - sizes[0] < 380 * 4 + 512
    for bad in ((30, 8, 128, 1, 3, 1, 1), (32, 8, 80, 1, 3, 1, 1), (32, 8, 128, 1, -1, 1, 1),
                (32, 8, 128, 1, 3, 0, 1), (32, 8, 128, 1, 3, 1, -1)):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_paged_shared_decode_workspace_bytes(*bad)
    for bad in ((30, 8, 128, 1, 3, 1), (32, 8, 128, 1, -3, 1), (32, 8, 128, 1, 3, -1)):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_paged_prefill_workspace_bytes(*bad)


def test_empty_calls_are_no_ops_and_need_no_arrays():
    none = dict(q=None, o=None, workspace=None, seq_lens=None, ws_bytes=0)
    assert call("gdn_paged_shared_decode", SHARED, dict(batch=0, group_cu=None, **none)) == 0
    assert call("gdn_paged_prefill", PREFILL, dict(n_seqs=0, **none)) == 0
    assert call("gdn_paged_prefill", PREFILL, dict(total_tokens=0, **none)) == 0
    assert call("gdn_paged_copy", COPY, dict(n=0, copy_src=None, copy_dst=None)) == 0
    assert call("gdn_paged_copy", COPY, dict(n_caches=0, caches=None)) == 0
    assert gdn.gdn_paged_prefill_workspace_bytes(32, 8, 128, 1, 0, 50) == 0
    assert gdn.gdn_paged_prefill_workspace_bytes(32, 8, 128, 1, 3, 0) == 0
    assert gdn.gdn_paged_shared_decode_workspace_bytes(32, 8, 128, 1, 0, 1, 2) == 0
    # the dimensions are looked at all the same
    assert call("gdn_paged_prefill", PREFILL, dict(n_seqs=0, dims=paged(d=80))) == UNSUPPORTED
    assert call("gdn_paged_copy", COPY, dict(n=0, page_bytes=8)) == UNSUPPORTED


def test_binding_refuses_tensors_off_the_gpu():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 4, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    for fn in (lambda: gdn.gdn_paged_fork(i, i, i, i.view(1, 1), 16, i, i),
               lambda: gdn.gdn_paged_free(i, i, i.view(1, 1), 16, i),
               lambda: gdn.gdn_paged_compact(i, i.view(1, 1), 16, i),
               lambda: gdn.gdn_paged_copy([cache], i, i),
               lambda: gdn.gdn_paged_prefill(q, cache, cache, i.view(1, 1), i, i),
               lambda: gdn.gdn_paged_shared_decode(q, cache, cache, i.view(1, 1), i, i, i)):
        with pytest.raises(ValueError, match="GPU"):
            fn()
