"""Refusals, sizes and no-ops of the paged attention entry points, on a host without a GPU: bad
arguments are turned down before any HIP call."""
import ctypes

import pytest

from gated_delta_rule_prefill_amd import gdn
from gated_delta_rule_prefill_amd.gdn import gdn_latent_dims_t, gdn_paged_dims_t

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


# ---------------------------------------------------------------------------------- plan
PLAN = dict(ctx_lens=FAKE, new_lens=FAKE + 64, n=4, block_size=64, block_table=FAKE, max_blocks=8,
            free_blocks=FAKE, n_free=9, max_tokens=100, cu_seqlens=FAKE, seq_lens=FAKE + 128,
            slot_map=FAKE, positions=FAKE, counts=FAKE, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(ctx_lens=None), NULL), (dict(new_lens=None), NULL), (dict(seq_lens=None), NULL),
    (dict(block_table=None), NULL), (dict(free_blocks=None), NULL), (dict(cu_seqlens=None), NULL),
    (dict(counts=None), NULL), (dict(slot_map=None), NULL), (dict(positions=None), NULL),
    (dict(n=0, counts=None), NULL), (dict(max_tokens=0, max_blocks=0, cu_seqlens=None), NULL),
    (dict(n=-1), SHAPE), (dict(block_size=0), SHAPE), (dict(block_size=-8), SHAPE),
    (dict(max_blocks=-1), SHAPE), (dict(n_free=-1), SHAPE), (dict(max_tokens=-1), SHAPE),
    (dict(seq_lens=FAKE), SHAPE), (dict(seq_lens=FAKE + 64), SHAPE),
    (dict(slot_map=FAKE + 8), ALIGN), (dict(positions=FAKE + 4), ALIGN),
    (dict(block_table=FAKE + 4), ALIGN), (dict(ctx_lens=FAKE + 4), ALIGN),
    (dict(free_blocks=FAKE + 2), ALIGN),
])
def test_plan_refuses(kw, status):
    refused(status, call("gdn_paged_plan", PLAN, kw))


# -------------------------------------------------------------------------------- append
APPEND = dict(dtype=1, k=FAKE, k_stride=512, v=FAKE, v_stride=512, slot_map=FAKE, tokens=3,
              kv_heads=4, d=128, k_cache=FAKE, v_cache=FAKE, n_blocks=10, block_size=16,
              stream=None)
LATENT_APPEND = dict(dtype=1, c=FAKE, c_stride=512, k_pe=FAKE, pe_stride=64, slot_map=FAKE,
                     tokens=3, rank=512, d_rope=64, cache=FAKE, n_blocks=10, block_size=16,
                     stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slot_map=None), NULL),
    (dict(k_cache=None), NULL), (dict(v_cache=None), NULL),
    (dict(k=FAKE + 8), ALIGN), (dict(v_cache=FAKE + 2), ALIGN), (dict(slot_map=FAKE + 4), ALIGN),
    (dict(k_stride=516), ALIGN), (dict(v_stride=513), ALIGN),
    (dict(dtype=0, k_stride=514, v_stride=512), ALIGN),
    (dict(k_stride=511), SHAPE), (dict(v_stride=0), SHAPE), (dict(k_stride=-512), SHAPE),
    (dict(tokens=-1), SHAPE), (dict(kv_heads=0), SHAPE), (dict(n_blocks=0), SHAPE),
    (dict(block_size=0), SHAPE),
    (dict(d=96), UNSUPPORTED), (dict(d=512), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(n_blocks=I32_MAX, block_size=2), UNSUPPORTED),
    (dict(n_blocks=1 << 20, block_size=1 << 10, kv_heads=4), UNSUPPORTED),
    (dict(kv_heads=1 << 18, k_stride=1 << 25, v_stride=1 << 25, n_blocks=1, block_size=1),
     UNSUPPORTED),
])
def test_append_refuses(kw, status):
    refused(status, call("gdn_paged_append", APPEND, kw))


@pytest.mark.parametrize("kw,status", [
    (dict(c=None), NULL), (dict(k_pe=None), NULL), (dict(slot_map=None), NULL),
    (dict(cache=None), NULL), (dict(c=FAKE + 8), ALIGN), (dict(cache=FAKE + 8), ALIGN),
    (dict(c_stride=516), ALIGN), (dict(pe_stride=68), ALIGN),
    (dict(c_stride=504), SHAPE), (dict(pe_stride=56), SHAPE), (dict(tokens=-1), SHAPE),
    (dict(n_blocks=0), SHAPE), (dict(block_size=-1), SHAPE),
    (dict(rank=12), UNSUPPORTED), (dict(rank=0), UNSUPPORTED), (dict(d_rope=4), UNSUPPORTED),
    (dict(rank=65544, c_stride=65544), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
    (dict(n_blocks=1 << 16, block_size=1 << 16), UNSUPPORTED),
])
def test_latent_append_refuses(kw, status):
    refused(status, call("gdn_latent_append", LATENT_APPEND, kw))


# -------------------------------------------------------------------------- paged decode
def paged(H=32, kv=8, d=128, dtype=1):
    return ctypes.byref(gdn_paged_dims_t(H, kv, d, dtype, 0.1))


DECODE = dict(dims=paged(), q=FAKE, k_cache=FAKE, v_cache=FAKE, n_blocks=100, block_size=16,
              block_table=FAKE, max_blocks=20, seq_lens=FAKE, batch=3, n_pos=1, o=FAKE,
              workspace=FAKE, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dims=None), NULL), (dict(q=None), NULL), (dict(k_cache=None), NULL),
    (dict(v_cache=None), NULL), (dict(block_table=None), NULL), (dict(seq_lens=None), NULL),
    (dict(o=None), NULL), (dict(workspace=None), NULL),
    (dict(q=FAKE + 8), ALIGN), (dict(v_cache=FAKE + 8), ALIGN), (dict(workspace=FAKE + 8), ALIGN),
    (dict(block_table=FAKE + 4), ALIGN), (dict(seq_lens=FAKE + 4), ALIGN),
    (dict(dims=paged(H=0)), SHAPE), (dict(dims=paged(kv=0)), SHAPE),
    (dict(dims=paged(H=30)), SHAPE), (dict(dims=paged(H=4, kv=8)), SHAPE),
    (dict(batch=-1), SHAPE), (dict(n_blocks=0), SHAPE), (dict(block_size=0), SHAPE),
    (dict(max_blocks=0), SHAPE),
    (dict(dims=paged(H=1032)), UNSUPPORTED), (dict(dims=paged(d=96)), UNSUPPORTED),
    (dict(dims=paged(dtype=2)), UNSUPPORTED), (dict(n_pos=0), UNSUPPORTED),
    (dict(n_pos=17), UNSUPPORTED), (dict(max_blocks=1 << 26), UNSUPPORTED),
    (dict(n_blocks=1 << 28), UNSUPPORTED), (dict(max_blocks=1 << 22, batch=1 << 8), UNSUPPORTED),
    (dict(ws_bytes=1000), WORKSPACE), (dict(ws_bytes=0), WORKSPACE),
])
def test_paged_decode_refuses(kw, status):
    refused(status, call("gdn_paged_decode", DECODE, kw))


def test_paged_decode_workspace_is_exact_and_does_not_depend_on_the_batch():
    args = (32, 8, 128, 1)
    need = gdn.gdn_paged_decode_workspace_bytes(*args, 3)
    assert call("gdn_paged_decode", DECODE, dict(ws_bytes=need - 1)) == WORKSPACE
    # two parts of a 16-row tile per worker; the notes of 3 x 8 units or of every worker on top
    sizes = [gdn.gdn_paged_decode_workspace_bytes(*args, b) for b in (1, 40, 10 ** 6)]
    assert max(sizes) - min(sizes) <= 1024 * 16
    assert gdn.gdn_paged_decode_workspace_bytes(*args, 0) == 0
    for bad in ((30, 8, 128, 1, 3), (32, 8, 80, 1, 3), (32, 8, 128, 1, -1), (32, 8, 128, 1, 3, 0)):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_paged_decode_workspace_bytes(*bad)
    assert gdn.load().gdn_paged_decode_workspace_bytes(paged(), 1, 1, None) == NULL


# -------------------------------------------------------------------------------- latent
def latent(H=16, rank=512, rope=64, dn=128, dv=128, dtype=1):
    return ctypes.byref(gdn_latent_dims_t(H, rank, rope, dn, dv, dtype, 0.1))


LATENT = dict(dims=latent(), q_nope=FAKE, q_pe=FAKE, w_kv=FAKE, cache=FAKE, n_blocks=100,
              block_size=16, block_table=FAKE, max_blocks=20, seq_lens=FAKE, batch=3, n_pos=1,
              o=FAKE, workspace=FAKE, ws_bytes=1 << 40, stream=None)
PREFILL = dict(dims=latent(), q_nope=FAKE, q_pe=FAKE, w_kv=FAKE, cache=FAKE, n_blocks=100,
               block_size=16, block_table=FAKE, max_blocks=20, cu_seqlens=FAKE, seq_lens=FAKE,
               n_seqs=3, total_tokens=50, total_keys=90, o=FAKE, workspace=FAKE,
               ws_bytes=1 << 40, stream=None)
BOTH = [
    (dict(dims=None), NULL), (dict(q_nope=None), NULL), (dict(q_pe=None), NULL),
    (dict(w_kv=None), NULL), (dict(cache=None), NULL), (dict(block_table=None), NULL),
    (dict(seq_lens=None), NULL), (dict(o=None), NULL), (dict(workspace=None), NULL),
    (dict(q_nope=FAKE + 8), ALIGN), (dict(w_kv=FAKE + 2), ALIGN), (dict(cache=FAKE + 8), ALIGN),
    (dict(dims=latent(H=0)), SHAPE), (dict(n_blocks=0), SHAPE), (dict(block_size=0), SHAPE),
    (dict(max_blocks=-3), SHAPE),
    (dict(dims=latent(H=1025)), UNSUPPORTED), (dict(dims=latent(rank=384)), UNSUPPORTED),
    (dict(dims=latent(rope=32)), UNSUPPORTED), (dict(dims=latent(dn=96, dv=96)), UNSUPPORTED),
    (dict(dims=latent(dv=64)), UNSUPPORTED), (dict(dims=latent(dtype=0)), UNSUPPORTED),
    (dict(max_blocks=1 << 26), UNSUPPORTED), (dict(n_blocks=1 << 28), UNSUPPORTED),
    (dict(ws_bytes=100), WORKSPACE),
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(batch=-1), SHAPE), (dict(n_pos=0), UNSUPPORTED), (dict(n_pos=17), UNSUPPORTED),
    (dict(batch=(1 << 20) + 1), UNSUPPORTED), (dict(batch=1 << 17, n_pos=9), UNSUPPORTED),
    (dict(max_blocks=1 << 22, batch=1 << 12), UNSUPPORTED),
])
def test_latent_decode_refuses(kw, status):
    refused(status, call("gdn_latent_decode", LATENT, kw))


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(cu_seqlens=None), NULL), (dict(cu_seqlens=FAKE + 4), ALIGN),
    (dict(n_seqs=-1), SHAPE), (dict(total_tokens=-1), SHAPE), (dict(total_keys=-1), SHAPE),
    (dict(total_keys=1 << 31), UNSUPPORTED), (dict(n_seqs=1 << 26), UNSUPPORTED),
    (dict(total_tokens=1 << 30), UNSUPPORTED),
])
def test_latent_prefill_refuses(kw, status):
    refused(status, call("gdn_latent_prefill", PREFILL, kw))


def test_latent_workspaces_are_exact():
    dims = (16, 512, 64, 128, 128)
    need = gdn.gdn_latent_decode_workspace_bytes(*dims, 3)
    assert call("gdn_latent_decode", LATENT, dict(ws_bytes=need - 1)) == WORKSPACE
    # per (request, head): the absorbed query (bf16) and the weighted latent (fp32)
    more = gdn.gdn_latent_decode_workspace_bytes(*dims, 259)
    assert 256 * 16 * 512 * 6 <= more - need <= 256 * 16 * 512 * 6 + 4096
    need = gdn.gdn_latent_prefill_workspace_bytes(*dims, 3, 50, 90)
    assert call("gdn_latent_prefill", PREFILL, dict(ws_bytes=need - 1)) == WORKSPACE
    # a key and a value per head and a rotary key, bf16, of each of 64000 more tokens
    per_token = (16 * 2 * 128 + 64) * 2 + 1
    more = gdn.gdn_latent_prefill_workspace_bytes(*dims, 3, 50, 64090)
    assert abs((more - need) / 64000 / per_token - 1) < 0.01
    assert gdn.gdn_latent_prefill_workspace_bytes(*dims, 0, 50, 90) == 0
    assert gdn.gdn_latent_prefill_workspace_bytes(*dims, 3, 0, 90) == 0
    assert gdn.gdn_latent_decode_workspace_bytes(*dims, 0) == 0
    with pytest.raises(gdn.GdnError):
        gdn.gdn_latent_decode_workspace_bytes(*dims, 1 << 21)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_latent_prefill_workspace_bytes(16, 512, 64, 128, 64, 3, 50, 90)


def test_empty_calls_are_no_ops_and_need_no_arrays():
    none = dict(q=None, o=None, workspace=None, seq_lens=None, ws_bytes=0)
    assert call("gdn_paged_decode", DECODE, dict(batch=0, **none)) == 0
    none = dict(q_nope=None, o=None, workspace=None, seq_lens=None, ws_bytes=0)
    assert call("gdn_latent_decode", LATENT, dict(batch=0, **none)) == 0
    assert call("gdn_latent_prefill", PREFILL, dict(n_seqs=0, **none)) == 0
    assert call("gdn_latent_prefill", PREFILL, dict(total_tokens=0, **none)) == 0
    assert call("gdn_paged_append", APPEND, dict(tokens=0, k=None, slot_map=None)) == 0
    assert call("gdn_latent_append", LATENT_APPEND, dict(tokens=0, c=None, cache=None)) == 0
    # the dimensions are looked at all the same
    assert call("gdn_paged_decode", DECODE, dict(batch=0, dims=paged(d=80))) == UNSUPPORTED
    assert call("gdn_paged_append", APPEND, dict(tokens=0, d=80)) == UNSUPPORTED


def test_binding_refuses_tensors_off_the_gpu():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 4, 16, 64, dtype=torch.bfloat16)
    ints = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_paged_decode(q, cache, cache, ints.view(1, 1), ints)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_paged_append(q, q, torch.zeros(1, dtype=torch.int64), cache, cache)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_paged_plan(ints, ints, ints.view(1, 1), ints, 16, 4)
