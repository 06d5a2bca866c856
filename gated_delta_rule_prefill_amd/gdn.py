"""Thin ctypes binding of libgdn.so (include/gdn.h). Argument marshalling only: every step
of the computation runs in the library's HIP kernels; there is no CPU fallback, and a
missing library raises.

Functions carry the C names. Tensors are torch CUDA (HIP) tensors; the HIP stream is the
current torch stream unless one is given.
"""
import contextlib
import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# GDN_LIB names another build of the same library (for instance one whose host code carries
# sanitizers); by default the in-tree libgdn.so
LIB_PATH = os.environ.get("GDN_LIB") or os.path.join(HERE, "libgdn.so")

GDN_DTYPE_F32, GDN_DTYPE_BF16 = 0, 1
# include/gdn.h GDN_COPY_MAX_CACHES: most pools of one gdn_paged_copy call
GDN_COPY_MAX_CACHES = 128
# include/gdn.h GDN_NOALLOC_SCRATCH_BYTES: the allocation-free prefill's per-GPU workspace
GDN_NOALLOC_SCRATCH_BYTES = 128 << 20
GDN_GATE_SCALAR, GDN_GATE_PER_KEY = 0, 1


class GdnError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed with status {status} ({msg})")
        self.status = status


class gdn_dims_t(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("gate", ctypes.c_int32), ("scale", ctypes.c_float),
                ("qk_l2norm", ctypes.c_int32)]


class gdn_deltalog_pool_t(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("lbar", ctypes.c_void_p), ("klog", ctypes.c_void_p),
                ("ulog", ctypes.c_void_p), ("lamlog", ctypes.c_void_p), ("len", ctypes.c_void_p),
                ("M", ctypes.c_int32)]


class gdn_paged_dims_t(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class gdn_latent_dims_t(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("d_rope", ctypes.c_int32), ("d_nope", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int32
_SZ = ctypes.c_size_t
_DIMS = ctypes.POINTER(gdn_dims_t)
_L = ctypes.c_int64
_POOL = ctypes.POINTER(gdn_deltalog_pool_t)
_PAGED = ctypes.POINTER(gdn_paged_dims_t)
_LATENT = ctypes.POINTER(gdn_latent_dims_t)

_SIGS = {
    "gdn_prefill_workspace_bytes": [_DIMS, _I, _I, _I, ctypes.POINTER(_SZ)],
    "gdn_prefill_chunked": [_DIMS, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _P, _P, _P, _P,
                            _SZ, _P],
    "gdn_prefill_chunked_ckpt": [_DIMS, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _P, _P,
                                 _P, _P, _P, _I, _P, _P, _SZ, _P],
    "gdn_prefill_chunked_conv": [_DIMS, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _P, _I, _P,
                                 _P, _P, _P, _SZ, _P],
    "gdn_prefill_chunked_noalloc": [_DIMS, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _P,
                                    _P, _P, _P],
    "gdn_decode_step": [_DIMS, _P, _P, _P, _P, _P, _P, _I, _P, _I, _P, _P],
    "gdn_decode_spec": [_DIMS, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _P, _P],
    "gdn_decode_fused": [_DIMS, _P, _P, _I, _P, _P, _P, _P, _P, ctypes.c_float, _P, _I, _P, _I,
                         _P, _P],
    "gdn_deltalog_workspace_bytes": [_DIMS, _I, _I, ctypes.POINTER(_SZ)],
    "gdn_decode_deltalog": [_DIMS, _P, _P, _P, _P, _P, _POOL, _I, _P, _I, _P, _P, _SZ, _P],
    "gdn_deltalog_reset": [_DIMS, _POOL, _I, _P, _I, _P],
    "gdn_deltalog_materialize": [_DIMS, _POOL, _I, _P, _I, _P],
    "gdn_conv1d_silu": [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P],
    "gdn_paged_plan": [_P, _P, _I, _I, _P, _I, _P, _I, _I, _P, _P, _P, _P, _P, _P],
    "gdn_paged_append": [_I, _P, _L, _P, _L, _P, _I, _I, _I, _P, _P, _I, _I, _P],
    "gdn_latent_append": [_I, _P, _L, _P, _L, _P, _I, _I, _I, _P, _I, _I, _P],
    "gdn_paged_fork": [_P, _P, _P, _I, _P, _I, _I, _I, _P, _I, _P, _I, _P, _P, _P, _P],
    "gdn_paged_free_workspace_bytes": [_I, ctypes.POINTER(_SZ)],
    "gdn_paged_free": [_P, _P, _I, _P, _I, _I, _I, _P, _I, _P, _I, _P, _P, _SZ, _P],
    "gdn_paged_compact_workspace_bytes": [_I, ctypes.POINTER(_SZ)],
    "gdn_paged_compact": [_P, _I, _P, _I, _I, _P, _I, _P, _P, _I, _P, _P, _SZ, _P],
    "gdn_paged_copy": [_P, _I, _L, _I, _P, _P, _I, _P, _P],
    "gdn_paged_shared_decode_workspace_bytes": [_PAGED, _I, _I, _I, ctypes.POINTER(_SZ)],
    "gdn_paged_shared_decode": [_PAGED, _P, _P, _P, _I, _I, _P, _I, _P, _I, _I, _P, _P, _I, _L, _P,
                                _P, _SZ, _P],
    "gdn_paged_prefill_workspace_bytes": [_PAGED, _I, _I, ctypes.POINTER(_SZ)],
    "gdn_paged_prefill": [_PAGED, _P, _P, _P, _I, _I, _P, _I, _P, _P, _I, _I, _P, _P, _SZ, _P],
    "gdn_paged_decode_workspace_bytes": [_PAGED, _I, _I, ctypes.POINTER(_SZ)],
    "gdn_paged_decode": [_PAGED, _P, _P, _P, _I, _I, _P, _I, _P, _I, _I, _P, _P, _SZ, _P],
    "gdn_latent_decode_workspace_bytes": [_LATENT, _I, _I, ctypes.POINTER(_SZ)],
    "gdn_latent_decode": [_LATENT, _P, _P, _P, _P, _I, _I, _P, _I, _P, _I, _I, _P, _P, _SZ, _P],
    "gdn_latent_prefill_workspace_bytes": [_LATENT, _I, _I, _L, ctypes.POINTER(_SZ)],
    "gdn_latent_prefill": [_LATENT, _P, _P, _P, _P, _I, _I, _P, _I, _P, _P, _I, _I, _L, _P, _P,
                           _SZ, _P],
    "gdn_status_string": [ctypes.c_int],
    "gdn_last_error": [],
    "gdn_abi_version": [],
}


def load(path: str = LIB_PATH):
    """Load libgdn.so (built in-tree by build_lib.py). Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise ImportError(f"{path} not found: build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(path)
        for name, args in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_last_error.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def lib():
    return load()


def gdn_status_string(status: int) -> str:
    return lib().gdn_status_string(int(status)).decode()


def gdn_last_error() -> str:
    return lib().gdn_last_error().decode()


def gdn_abi_version() -> int:
    return int(lib().gdn_abi_version())


def _check(fn, status):
    if status != 0:
        raise GdnError(fn, status, gdn_last_error() or gdn_status_string(status))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return GDN_DTYPE_BF16
    if t.dtype == torch.float32:
        return GDN_DTYPE_F32
    raise TypeError(f"q/k/v must be fp32 or bf16, got {t.dtype}")


def _dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("all tensors must be on the GPU")
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")


def make_dims(H, dk, dv, dtype_code, perkey, scale, qk_l2norm):
    return gdn_dims_t(int(H), int(dk), int(dv), int(dtype_code),
                      GDN_GATE_PER_KEY if perkey else GDN_GATE_SCALAR, float(scale),
                      1 if qk_l2norm else 0)


# ---------------------------------------------------------------------------- prefill
def gdn_prefill_workspace_bytes(H, dk, dv, dtype, perkey, n_seqs, total_tokens, chunk):
    dims = make_dims(H, dk, dv, dtype if isinstance(dtype, int) else
                     (GDN_DTYPE_BF16 if dtype == torch.bfloat16 else GDN_DTYPE_F32),
                     perkey, 1.0, False)
    out = _SZ(0)
    _check("gdn_prefill_workspace_bytes",
           lib().gdn_prefill_workspace_bytes(ctypes.byref(dims), int(n_seqs), int(total_tokens),
                                             int(chunk), ctypes.byref(out)))
    return int(out.value)


def gdn_prefill_chunked(q, k, v, g, beta, cu_seqlens, chunk, state_pool, slots, has_init=None,
                        scale=1.0, qk_l2norm=False, o=None, workspace=None, stream=None):
    """Chunked prefill. q, k [T,H,dk]; v [T,H,dv]; g [T,H] or [T,H,dk] fp32; beta [T,H] fp32;
    cu_seqlens [n+1] int32; state_pool [slots,H,dk,dv] fp32 (updated in place);
    slots [n] int32; has_init [n] int32 or None. Returns o [T,H,dv]."""
    T, H, dk = q.shape
    dv = v.shape[2]
    n = cu_seqlens.numel() - 1
    perkey = g.dim() == 3
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    need = gdn_prefill_workspace_bytes(H, dk, dv, _dtype_code(q), perkey, n, T, chunk)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _dev(q, k, v, g, beta, cu_seqlens, state_pool, slots, has_init, o, workspace)
    dims = make_dims(H, dk, dv, _dtype_code(q), perkey, scale, qk_l2norm)
    _check("gdn_prefill_chunked", lib().gdn_prefill_chunked(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
        int(n), int(T), int(chunk), _ptr(state_pool), int(state_pool.shape[0]), _ptr(slots),
        _ptr(has_init), _ptr(o), _ptr(workspace), int(workspace.numel()), _stream(stream)))
    return o


def gdn_prefill_chunked_noalloc(q, k, v, g, beta, cu_seqlens, chunk, state_pool, slots,
                                has_init=None, scale=1.0, qk_l2norm=False, o=None,
                                stream=None):
    """gdn_prefill_chunked without a workspace: the library's per-GPU scratch array serves
    as one (at most GDN_NOALLOC_SCRATCH_BYTES). Nothing is allocated when `o` is given.
    Arguments as gdn_prefill_chunked. Returns o."""
    T, H, dk = q.shape
    dv = v.shape[2]
    n = cu_seqlens.numel() - 1
    perkey = g.dim() == 3
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    _dev(q, k, v, g, beta, cu_seqlens, state_pool, slots, has_init, o)
    dims = make_dims(H, dk, dv, _dtype_code(q), perkey, scale, qk_l2norm)
    _check("gdn_prefill_chunked_noalloc", lib().gdn_prefill_chunked_noalloc(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
        int(n), int(T), int(chunk), _ptr(state_pool), int(state_pool.shape[0]), _ptr(slots),
        _ptr(has_init), _ptr(o), _stream(stream)))
    return o


def gdn_prefill_chunked_ckpt(q, k, v, g, beta, cu_seqlens, chunk, state_pool, slots,
                             ckpt_cu, ckpt_pos, ckpt_slots, has_init=None, scale=1.0,
                             qk_l2norm=False, o=None, workspace=None, stream=None):
    """Chunked prefill that also writes the state after ckpt_pos[i] tokens of its sequence
    into pool slot ckpt_slots[i]; the entries of sequence n are ckpt_cu[n]:ckpt_cu[n+1]
    (all three int32 device tensors). Other arguments as gdn_prefill_chunked. Returns o."""
    T, H, dk = q.shape
    dv = v.shape[2]
    n = cu_seqlens.numel() - 1
    perkey = g.dim() == 3
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    need = gdn_prefill_workspace_bytes(H, dk, dv, _dtype_code(q), perkey, n, T, chunk)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _dev(q, k, v, g, beta, cu_seqlens, state_pool, slots, has_init, ckpt_cu, ckpt_pos,
         ckpt_slots, o, workspace)
    dims = make_dims(H, dk, dv, _dtype_code(q), perkey, scale, qk_l2norm)
    _check("gdn_prefill_chunked_ckpt", lib().gdn_prefill_chunked_ckpt(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
        int(n), int(T), int(chunk), _ptr(state_pool), int(state_pool.shape[0]), _ptr(slots),
        _ptr(has_init), _ptr(ckpt_cu), _ptr(ckpt_pos), _ptr(ckpt_slots), int(ckpt_pos.numel()),
        _ptr(o), _ptr(workspace), int(workspace.numel()), _stream(stream)))
    return o


def gdn_prefill_chunked_conv(x, conv_w, g, beta, cu_seqlens, chunk, state_pool, slots,
                             conv_state=None, has_init=None, scale=1.0, qk_l2norm=False,
                             o=None, workspace=None, stream=None):
    """Chunked prefill with the short convolution and SiLU fused into its loads.
    x [T, 3 H d] raw q|k|v projection; conv_w [3 H d, W] fp32; conv_state [slots, 3 H d, W-1]
    (x's dtype) or None: read as the history of sequences with has_init and overwritten with
    each sequence's last W-1 rows. g [T,H] or [T,H,d]; other arguments as
    gdn_prefill_chunked. Returns o [T, H, d]."""
    T = x.shape[0]
    H = beta.shape[1]
    d = x.shape[1] // (3 * H)
    W = conv_w.shape[1]
    n = cu_seqlens.numel() - 1
    perkey = g.dim() == 3
    if o is None:
        o = torch.empty((T, H, d), dtype=x.dtype, device=x.device)
    need = gdn_prefill_workspace_bytes(H, d, d, _dtype_code(x), perkey, n, T, chunk)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _dev(x, conv_w, conv_state, g, beta, cu_seqlens, state_pool, slots, has_init, o, workspace)
    dims = make_dims(H, d, d, _dtype_code(x), perkey, scale, qk_l2norm)
    _check("gdn_prefill_chunked_conv", lib().gdn_prefill_chunked_conv(
        ctypes.byref(dims), _ptr(x), _ptr(conv_w), int(W), _ptr(conv_state), _ptr(g),
        _ptr(beta), _ptr(cu_seqlens), int(n), int(T), int(chunk), _ptr(state_pool),
        int(state_pool.shape[0]), _ptr(slots), _ptr(has_init), _ptr(o), _ptr(workspace),
        int(workspace.numel()), _stream(stream)))
    return o


# ----------------------------------------------------------------------------- decode
def gdn_decode_step(q, k, v, g, beta, state_pool, slots, scale=1.0, qk_l2norm=False, o=None,
                    stream=None):
    """One decode step. q, k [B,H,dk]; v [B,H,dv]; g [B,H] or [B,H,dk]; beta [B,H];
    state_pool [slots,H,dk,dv] fp32 updated in place; slots [B] int32. Returns o."""
    B, H, dk = q.shape
    dv = v.shape[2]
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    _dev(q, k, v, g, beta, state_pool, slots, o)
    dims = make_dims(H, dk, dv, _dtype_code(q), g.dim() == 3, scale, qk_l2norm)
    _check("gdn_decode_step", lib().gdn_decode_step(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_pool),
        int(state_pool.shape[0]), _ptr(slots), int(B), _ptr(o), _stream(stream)))
    return o


# --------------------------------------------------------------------------- DeltaLog
def gdn_decode_spec(q, k, v, g, beta, state_pool, spec_slots, num_accepted, scale=1.0,
                    qk_l2norm=False, o=None, stream=None):
    """Speculative-decoding verify step. q, k [B,P,H,dk]; v [B,P,H,dv]; g [B,P,H] or
    [B,P,H,dk] fp32; beta [B,P,H] fp32; state_pool [slots,H,dk,dv] fp32; spec_slots [B,P]
    int32; num_accepted [B] int32. Returns o [B,P,H,dv]."""
    B, P, H, dk = q.shape
    dv = v.shape[3]
    perkey = g.dim() == 4
    if o is None:
        o = torch.empty((B, P, H, dv), dtype=q.dtype, device=q.device)
    _dev(q, k, v, g, beta, state_pool, spec_slots, num_accepted, o)
    dims = make_dims(H, dk, dv, _dtype_code(q), perkey, scale, qk_l2norm)
    _check("gdn_decode_spec", lib().gdn_decode_spec(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_pool),
        int(state_pool.shape[0]), _ptr(spec_slots), _ptr(num_accepted), int(B), int(P), _ptr(o),
        _stream(stream)))
    return o


def gdn_decode_fused(x, conv_w, conv_state, forget_b, write_logit, A_log, dt_bias, lower_bound,
                     state_pool, slots, scale=1.0, qk_l2norm=True, o=None, stream=None):
    """Fused KDA decode step. x [B, 3 H d] (q|k|v before the convolution); conv_w [3 H d, W]
    fp32; conv_state [slots, 3 H d, W-1] (x's dtype, updated in place); forget_b [B, H, d],
    write_logit [B, H], A_log [H], dt_bias [H, d] fp32; state_pool [slots, H, d, d] fp32;
    slots [B] int32. Returns o [B, H, d]."""
    B, H, dk = forget_b.shape
    W = conv_w.shape[1]
    if o is None:
        o = torch.empty((B, H, dk), dtype=x.dtype, device=x.device)
    _dev(x, conv_w, conv_state, forget_b, write_logit, A_log, dt_bias, state_pool, slots, o)
    dims = make_dims(H, dk, dk, _dtype_code(x), True, scale, qk_l2norm)
    _check("gdn_decode_fused", lib().gdn_decode_fused(
        ctypes.byref(dims), _ptr(x), _ptr(conv_w), int(W), _ptr(conv_state), _ptr(forget_b),
        _ptr(write_logit), _ptr(A_log), _ptr(dt_bias), float(lower_bound), _ptr(state_pool),
        int(state_pool.shape[0]), _ptr(slots), int(B), _ptr(o), _stream(stream)))
    return o


class DeltaLogPool:
    """Device buffers of a DeltaLog state pool (layouts of gdn_deltalog_pool_t)."""

    def __init__(self, base, M, perkey=False):
        n_slots, H, dk, dv = base.shape
        C = M - 1
        dl = (dk,) if perkey else ()
        dev = base.device
        self.base = base
        self.M = int(M)
        self.perkey = bool(perkey)
        self.lbar = torch.zeros((n_slots, H, *dl), dtype=torch.float32, device=dev)
        self.klog = torch.zeros((n_slots, H, C, dk), dtype=torch.int16, device=dev)
        self.ulog = torch.zeros((n_slots, H, C, dv), dtype=torch.float32, device=dev)
        self.lamlog = torch.zeros((n_slots, H, C, *dl), dtype=torch.float32, device=dev)
        self.len = torch.zeros((n_slots, H), dtype=torch.int32, device=dev)

    @property
    def n_slots(self):
        return int(self.base.shape[0])

    def struct(self):
        _dev(self.base, self.lbar, self.klog, self.ulog, self.lamlog, self.len)
        return gdn_deltalog_pool_t(self.base.data_ptr(), self.lbar.data_ptr(),
                                   self.klog.data_ptr(), self.ulog.data_ptr(),
                                   self.lamlog.data_ptr(), self.len.data_ptr(), self.M)


def gdn_deltalog_workspace_bytes(H, dk, dv, dtype, batch, M):
    dims = make_dims(H, dk, dv, dtype, False, 1.0, False)
    out = _SZ(0)
    _check("gdn_deltalog_workspace_bytes", lib().gdn_deltalog_workspace_bytes(
        ctypes.byref(dims), int(batch), int(M), ctypes.byref(out)))
    return int(out.value)


def gdn_decode_deltalog(q, k, v, g, beta, pool: DeltaLogPool, slots, scale=1.0,
                        qk_l2norm=False, o=None, stream=None):
    B, H, dk = q.shape
    dv = v.shape[2]
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    _dev(q, k, v, g, beta, slots, o)
    if (g.dim() == 3) != pool.perkey:
        raise ValueError("gate kind does not match the DeltaLog pool layout")
    dims = make_dims(H, dk, dv, _dtype_code(q), g.dim() == 3, scale, qk_l2norm)
    ps = pool.struct()
    _check("gdn_decode_deltalog", lib().gdn_decode_deltalog(
        ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), ctypes.byref(ps),
        pool.n_slots, _ptr(slots), int(B), _ptr(o), None, 0, _stream(stream)))
    return o


def _dl_maint(name, pool, slots, stream):
    n_slots, H, dk, dv = pool.base.shape
    dims = make_dims(H, dk, dv, GDN_DTYPE_F32, pool.perkey, 1.0, False)
    _dev(slots)
    ps = pool.struct()
    _check(name, getattr(lib(), name)(ctypes.byref(dims), ctypes.byref(ps), pool.n_slots,
                                      _ptr(slots), int(slots.numel()), _stream(stream)))


def gdn_deltalog_reset(pool: DeltaLogPool, slots, stream=None):
    _dl_maint("gdn_deltalog_reset", pool, slots, stream)


def gdn_deltalog_materialize(pool: DeltaLogPool, slots, stream=None):
    _dl_maint("gdn_deltalog_materialize", pool, slots, stream)


# ----------------------------------------------------------------------------- conv1d
def gdn_conv1d_silu(x, w, cu_seqlens, planes=1, y=None, stream=None):
    """x [T, channels]; w [channels, width] fp32. Returns y [planes, T, channels/planes]."""
    T, ch = x.shape
    if y is None:
        y = torch.empty((planes, T, ch // planes), dtype=x.dtype, device=x.device)
    _dev(x, w, cu_seqlens, y)
    _check("gdn_conv1d_silu", lib().gdn_conv1d_silu(
        _ptr(x), _ptr(w), _ptr(cu_seqlens), int(cu_seqlens.numel() - 1), int(T), int(ch),
        int(w.shape[1]), int(planes), _dtype_code(x), _ptr(y), _stream(stream)))
    return y


# ------------------------------------------------- paged softmax attention (hybrid models)
# These calls are short (a decode step's bookkeeping runs 4 us on the GPU), so the checks are
# kept to a few attribute reads per tensor; a failed one works out its message afterwards.
# Private names save 1.2 us a call; a torch without a GPU backend lacks them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",  # handle of a device's current stream
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_I32, _I64, _BF16 = torch.int32, torch.int64, torch.bfloat16


def _bad(name, t, shape, dtype):
    if not t.is_cuda:
        raise ValueError(f"all tensors must be on the GPU ({name} is on {t.device})")
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"all tensors must be contiguous ({name} is not)")
    raise ValueError(f"all tensors must be on one GPU ({name} is on {t.device})")


def _arg(name, t, shape, dtype, dev):
    """Address of a contiguous tensor of this shape and type on GPU `dev`."""
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != dev
            or not t.is_contiguous()):
        _bad(name, t, shape, dtype)
    return t.data_ptr()


def _table_arg(t, n, dev):
    if t.dim() != 2:
        raise ValueError("block_table must be [requests, max_blocks]")
    return _arg("block_table", t, (n, t.shape[1]), _I32, dev)


def _rows_arg(name, t, shape, dtype, dev):
    """Address and row stride (elements) of a token-major source whose rows may lie apart, as
    parts of a fused projection's output do."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _bad(name, t, shape, dtype)
    row = shape[1] * shape[2] if len(shape) == 3 else shape[1]
    if t.is_contiguous():
        return t.data_ptr(), row
    stride = t.stride()
    if stride[-1] != 1 or (len(shape) == 3 and shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError(f"{name}: each token's row must be contiguous")
    return t.data_ptr(), stride[0] if shape[0] > 1 else row


def _space(workspace, need, like, stream, dev):
    """Address and size of the workspace; one is allocated unless given."""
    if workspace is None:
        with torch.cuda.device(dev) if _current_device() != dev else contextlib.nullcontext():
            size = need()  # (the sizes go with the current GPU's CU count)
        workspace = _new((max(size, 1),), torch.uint8, like, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _bad("workspace", workspace, workspace.shape, workspace.dtype)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _new(shape, dtype, like, stream):
    """A buffer on the tensors' GPU. For a stream that is given it comes from that stream's
    memory, which work queued on the current stream cannot still be using, and is marked as used
    on the current stream too, where results are read as a rule."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    if not hasattr(stream, "cuda_stream"):
        # (handle 0 is the default stream; ExternalStream would take some other one for it)
        stream = (torch.cuda.ExternalStream(int(stream), device=like.device) if int(stream)
                  else torch.cuda.default_stream(like.device))
    now = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(now)
    return t


def _gpu(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("all tensors must be on the GPU")
    return dev


def _run(name, dev, stream, *args):
    """One call with the tensors' GPU current, on its current stream unless one is given."""
    if stream is None:
        handle = _raw_stream(dev)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    fn = getattr(lib(), name)
    if _current_device() == dev:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status:
        _check(name, status)


def gdn_paged_plan(ctx_lens, new_lens, block_table, free_blocks, block_size, max_tokens,
                   cu_seqlens=None, seq_lens=None, slot_map=None, positions=None, counts=None,
                   stream=None):
    """Bookkeeping of one step over a paged cache, on the GPU. ctx_lens, new_lens [n] int32;
    block_table [n, max_blocks] int32, updated in place; free_blocks [n_free] int32; max_tokens
    is the length of the token buffers. Returns (cu_seqlens [n + 1] int32, seq_lens [n] int32,
    slot_map [max_tokens] int64, positions [max_tokens] int32, counts [2] int32: tokens, pages
    asked for)."""
    n, T = ctx_lens.numel(), int(max_tokens)
    n_free = free_blocks.numel()
    if T < 0:
        raise ValueError("max_tokens must be >= 0")
    dev = _gpu(ctx_lens)
    like = ctx_lens
    cu_seqlens = _new((n + 1,), _I32, like, stream) if cu_seqlens is None else cu_seqlens
    seq_lens = _new((n,), _I32, like, stream) if seq_lens is None else seq_lens
    slot_map = _new((T,), _I64, like, stream) if slot_map is None else slot_map
    positions = _new((T,), _I32, like, stream) if positions is None else positions
    counts = _new((2,), _I32, like, stream) if counts is None else counts
    _run("gdn_paged_plan", dev, stream, _arg("ctx_lens", ctx_lens, (n,), _I32, dev),
         _arg("new_lens", new_lens, (n,), _I32, dev), n, int(block_size),
         _table_arg(block_table, n, dev), block_table.shape[1],
         _arg("free_blocks", free_blocks, (n_free,), _I32, dev), n_free, T,
         _arg("cu_seqlens", cu_seqlens, (n + 1,), _I32, dev),
         _arg("seq_lens", seq_lens, (n,), _I32, dev), _arg("slot_map", slot_map, (T,), _I64, dev),
         _arg("positions", positions, (T,), _I32, dev), _arg("counts", counts, (2,), _I32, dev))
    return cu_seqlens, seq_lens, slot_map, positions, counts


def gdn_paged_append(k, v, slot_map, k_cache, v_cache, stream=None):
    """Rows of new tokens into the cache. k, v [T, kv_heads, d] (tokens may lie apart, as parts
    of a fused projection); slot_map [T] int64; k_cache, v_cache [n_blocks, kv_heads,
    block_size, d], updated in place."""
    T, h, d = k.shape
    n_blocks, _, bs, _ = k_cache.shape
    dt, dev = k.dtype, _gpu(k_cache)
    ka, ks = _rows_arg("k", k, (T, h, d), dt, dev)
    va, vs = _rows_arg("v", v, (T, h, d), dt, dev)
    _run("gdn_paged_append", dev, stream, _dtype_code(k), ka, ks, va, vs,
         _arg("slot_map", slot_map, (T,), _I64, dev), T, h, d,
         _arg("k_cache", k_cache, (n_blocks, h, bs, d), dt, dev),
         _arg("v_cache", v_cache, (n_blocks, h, bs, d), dt, dev), n_blocks, bs)


def gdn_latent_append(c_kv, k_pe, slot_map, cache, stream=None):
    """Rows of new tokens into a latent cache. c_kv [T, rank], k_pe [T, d_rope] (rows may lie
    apart); slot_map [T] int64; cache [n_blocks, block_size, rank + d_rope], updated in
    place."""
    T, rank = c_kv.shape
    rope = k_pe.shape[1]
    n_blocks, bs, _ = cache.shape
    dt, dev = c_kv.dtype, _gpu(cache)
    ca, cs = _rows_arg("c_kv", c_kv, (T, rank), dt, dev)
    pa, ps = _rows_arg("k_pe", k_pe, (T, rope), dt, dev)
    _run("gdn_latent_append", dev, stream, _dtype_code(c_kv), ca, cs, pa, ps,
         _arg("slot_map", slot_map, (T,), _I64, dev), T, rank, rope,
         _arg("cache", cache, (n_blocks, bs, rank + rope), dt, dev), n_blocks, bs)


def _code(dtype):
    if isinstance(dtype, int):
        return dtype
    return _dtype_code(torch.empty(0, dtype=dtype))


def gdn_paged_decode_workspace_bytes(H, kv_heads, d, dtype, batch, n_pos=1):
    dims = gdn_paged_dims_t(int(H), int(kv_heads), int(d), _code(dtype), 1.0)
    out = _SZ(0)
    _check("gdn_paged_decode_workspace_bytes", lib().gdn_paged_decode_workspace_bytes(
        ctypes.byref(dims), int(batch), int(n_pos), ctypes.byref(out)))
    return int(out.value)


def gdn_paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale=1.0, o=None,
                     workspace=None, stream=None):
    """Attention of the newest tokens over a paged cache. q [B, H, d] (a decode step) or
    [B, P, H, d] (a verify step: the request's newest P tokens, all of them in the cache);
    k_cache, v_cache [n_blocks, kv_heads, block_size, d]; block_table [B, max_blocks] int32;
    seq_lens [B] int32. Returns o, shaped as q."""
    shape, dt = q.shape, q.dtype
    if len(shape) == 3:  # one position per request
        (B, H, d), P = shape, 1
    else:
        B, P, H, d = shape
    n_blocks, kv, bs, _ = k_cache.shape
    dev = _gpu(q)
    code = _dtype_code(q)
    o = _new(shape, dt, q, stream) if o is None else o
    ws, ws_bytes = _space(workspace, lambda: gdn_paged_decode_workspace_bytes(
        H, kv, d, code, B, P), q, stream, dev)
    _run("gdn_paged_decode", dev, stream, gdn_paged_dims_t(H, kv, d, code, scale),
         _arg("q", q, shape, dt, dev), _arg("k_cache", k_cache, (n_blocks, kv, bs, d), dt, dev),
         _arg("v_cache", v_cache, (n_blocks, kv, bs, d), dt, dev), n_blocks, bs,
         _table_arg(block_table, B, dev), block_table.shape[1],
         _arg("seq_lens", seq_lens, (B,), _I32, dev), B, P, _arg("o", o, shape, dt, dev), ws,
         ws_bytes)
    return o


def _table_rows(t, dev):
    """Address and shape of a table of which some rows are named."""
    return _table_arg(t, t.shape[0], dev), t.shape[0], t.shape[1]


def _pool_args(shares, dev):
    return _arg("shares", shares, (shares.numel(),), _I32, dev), shares.numel()


def gdn_paged_fork(src_rows, dst_rows, fork_lens, block_table, block_size, shares, free_blocks,
                   copy_src=None, copy_dst=None, counts=None, stream=None):
    """Requests that continue others: row dst_rows[i] of the table gets the first fork_lens[i]
    tokens of row src_rows[i] ([n] int32 each), sharing the whole pages (shares [n_blocks] int32
    counts a page's holders beyond the first) and taking a page of free_blocks for the rest.
    block_table [rows, max_blocks] int32 and shares are updated in place. Returns (copy_src [n],
    copy_dst [n]: pages to copy with gdn_paged_copy, -1 for none; counts [2]: pages asked of the
    free list, pages handed out)."""
    n, dev = src_rows.numel(), _gpu(block_table)
    n_free = free_blocks.numel()
    copy_src = _new((n,), _I32, block_table, stream) if copy_src is None else copy_src
    copy_dst = _new((n,), _I32, block_table, stream) if copy_dst is None else copy_dst
    counts = _new((2,), _I32, block_table, stream) if counts is None else counts
    _run("gdn_paged_fork", dev, stream, _arg("src_rows", src_rows, (n,), _I32, dev),
         _arg("dst_rows", dst_rows, (n,), _I32, dev), _arg("fork_lens", fork_lens, (n,), _I32, dev),
         n, *_table_rows(block_table, dev), int(block_size), *_pool_args(shares, dev),
         _arg("free_blocks", free_blocks, (n_free,), _I32, dev), n_free,
         _arg("copy_src", copy_src, (n,), _I32, dev), _arg("copy_dst", copy_dst, (n,), _I32, dev),
         _arg("counts", counts, (2,), _I32, dev))
    return copy_src, copy_dst, counts


def _bytes_of(name, *args):
    out = _SZ(0)
    _check(name, getattr(lib(), name)(*args, ctypes.byref(out)))
    return int(out.value)


def gdn_paged_free_workspace_bytes(n_blocks):
    return _bytes_of("gdn_paged_free_workspace_bytes", int(n_blocks))


def gdn_paged_free(rows, lens, block_table, block_size, shares, freed=None, max_freed=None,
                   counts=None, workspace=None, stream=None):
    """Requests that end: the pages of rows[i] ([n] int32) of the table for lens[i] tokens have a
    holder less, their entries become -1. Returns (freed [max_freed] int32: the pages that nobody
    holds any more in the order of their ids, then -1; counts [1]: how many). max_freed is by
    default as many as the rows can hold; `freed` may be a part of a longer list."""
    n, dev = rows.numel(), _gpu(block_table)
    if freed is None:
        most = min(n * block_table.shape[1], shares.numel()) if max_freed is None else max_freed
        freed = _new((int(most),), _I32, block_table, stream)
    counts = _new((1,), _I32, block_table, stream) if counts is None else counts
    ws, ws_bytes = _space(workspace, lambda: gdn_paged_free_workspace_bytes(shares.numel()),
                          block_table, stream, dev)
    most = freed.numel()
    _run("gdn_paged_free", dev, stream, _arg("rows", rows, (n,), _I32, dev),
         _arg("lens", lens, (n,), _I32, dev), n, *_table_rows(block_table, dev), int(block_size),
         *_pool_args(shares, dev), _arg("freed", freed, (most,), _I32, dev), most,
         _arg("counts", counts, (1,), _I32, dev), ws, ws_bytes)
    return freed, counts


def gdn_paged_compact_workspace_bytes(n_blocks):
    return _bytes_of("gdn_paged_compact_workspace_bytes", int(n_blocks))


def gdn_paged_compact(seq_lens, block_table, block_size, shares, max_copies=None, copy_src=None,
                      copy_dst=None, counts=None, workspace=None, stream=None):
    """Moves the live pages (those that the table's rows hold for seq_lens [rows] int32 tokens) to
    the front of the pool. block_table [rows, max_blocks] and shares [n_blocks] are updated in
    place. Returns (copy_src, copy_dst [max_copies] int32: the moves, to be made in every cache
    with gdn_paged_copy, then -1; counts [2]: live pages, moves). max_copies is by default as many
    as there can be."""
    n, dev = seq_lens.numel(), _gpu(block_table)
    if max_copies is None:
        max_copies = shares.numel() // 2 if copy_src is None else copy_src.numel()
    m = int(max_copies)
    copy_src = _new((m,), _I32, block_table, stream) if copy_src is None else copy_src
    copy_dst = _new((m,), _I32, block_table, stream) if copy_dst is None else copy_dst
    counts = _new((2,), _I32, block_table, stream) if counts is None else counts
    ws, ws_bytes = _space(workspace, lambda: gdn_paged_compact_workspace_bytes(shares.numel()),
                          block_table, stream, dev)
    _run("gdn_paged_compact", dev, stream, _arg("seq_lens", seq_lens, (n,), _I32, dev), n,
         _table_arg(block_table, n, dev), block_table.shape[1], int(block_size),
         *_pool_args(shares, dev), _arg("copy_src", copy_src, (m,), _I32, dev),
         _arg("copy_dst", copy_dst, (m,), _I32, dev), m, _arg("counts", counts, (2,), _I32, dev),
         ws, ws_bytes)
    return copy_src, copy_dst, counts


def gdn_paged_copy(caches, copy_src, copy_dst, count=None, stream=None):
    """Pages copy_src[i] copied to pages copy_dst[i] ([n] int32; -1, or the same: none) within each of
    the caches: contiguous tensors of one length (pages) and one number of bytes a page, of any type
    and shape (key, value and latent caches, state pools), GDN_COPY_MAX_CACHES of them at most. count
    [1] int32 on the GPU, or None: pairs from it on are not looked at."""
    n, dev = copy_src.numel(), _gpu(copy_src)
    addresses, like = [], None
    for c in caches:
        now = (c.shape[0], c.numel() // max(c.shape[0], 1) * c.element_size())
        like = now if like is None else like
        if now != like or c.get_device() != dev or not c.is_contiguous():
            raise ValueError("caches must be contiguous, on one GPU, and alike in their pages: got "
                             f"{tuple(c.shape)} {c.dtype} on {c.device}")
        addresses.append(c.data_ptr())
    if like is None:
        return
    count = None if count is None else _arg("count", count, (1,), _I32, dev)
    _run("gdn_paged_copy", dev, stream, (_P * len(addresses))(*addresses), len(addresses), like[1],
         like[0], _arg("copy_src", copy_src, (n,), _I32, dev),
         _arg("copy_dst", copy_dst, (n,), _I32, dev), n, count)


def gdn_paged_shared_decode_workspace_bytes(H, kv_heads, d, dtype, batch, n_pos, n_groups):
    dims = gdn_paged_dims_t(int(H), int(kv_heads), int(d), _code(dtype), 1.0)
    return _bytes_of("gdn_paged_shared_decode_workspace_bytes", ctypes.byref(dims), int(batch),
                     int(n_pos), int(n_groups))


def gdn_paged_shared_decode(q, k_cache, v_cache, block_table, seq_lens, group_cu, prefix_lens,
                            scale=1.0, min_bytes=-1, o=None, workspace=None, stream=None):
    """gdn_paged_decode for a batch in which groups of requests share a prefix, read once for the
    group: requests group_cu[g] .. group_cu[g + 1] - 1 ([groups + 1] int32) hold the same pages for
    their first prefix_lens[g] tokens ([groups] int32), or fewer of them, or have ended. Where that spares less than min_bytes of
    reads (negative: the library's rule) each request reads its own. Returns o, shaped as q."""
    shape, dt = q.shape, q.dtype
    if len(shape) == 3:  # one position per request
        (B, H, d), P = shape, 1
    else:
        B, P, H, d = shape
    n_blocks, kv, bs, _ = k_cache.shape
    groups = prefix_lens.numel()
    dev = _gpu(q)
    code = _dtype_code(q)
    o = _new(shape, dt, q, stream) if o is None else o
    ws, ws_bytes = _space(workspace, lambda: gdn_paged_shared_decode_workspace_bytes(
        H, kv, d, code, B, P, groups), q, stream, dev)
    _run("gdn_paged_shared_decode", dev, stream, gdn_paged_dims_t(H, kv, d, code, scale),
         _arg("q", q, shape, dt, dev), _arg("k_cache", k_cache, (n_blocks, kv, bs, d), dt, dev),
         _arg("v_cache", v_cache, (n_blocks, kv, bs, d), dt, dev), n_blocks, bs,
         _table_arg(block_table, B, dev), block_table.shape[1],
         _arg("seq_lens", seq_lens, (B,), _I32, dev), B, P,
         _arg("group_cu", group_cu, (groups + 1,), _I32, dev),
         _arg("prefix_lens", prefix_lens, (groups,), _I32, dev), groups, int(min_bytes),
         _arg("o", o, shape, dt, dev), ws, ws_bytes)
    return o


def gdn_paged_prefill_workspace_bytes(H, kv_heads, d, dtype, n_seqs, total_tokens):
    dims = gdn_paged_dims_t(int(H), int(kv_heads), int(d), _code(dtype), 1.0)
    return _bytes_of("gdn_paged_prefill_workspace_bytes", ctypes.byref(dims), int(n_seqs),
                     int(total_tokens))


def gdn_paged_prefill(q, k_cache, v_cache, block_table, cu_seqlens, seq_lens, scale=1.0, o=None,
                      workspace=None, stream=None):
    """Attention of packed new tokens over a paged cache that already holds them, causal. q
    [T, H, d]; k_cache, v_cache [n_blocks, kv_heads, block_size, d]; block_table [n, max_blocks]
    int32; cu_seqlens [n + 1] int32; seq_lens [n] int32, the new tokens included. Returns o
    [T, H, d]."""
    T, H, d = q.shape
    n = seq_lens.numel()
    n_blocks, kv, bs, _ = k_cache.shape
    dt, dev = q.dtype, _gpu(q)
    code = _dtype_code(q)
    o = _new((T, H, d), dt, q, stream) if o is None else o
    ws, ws_bytes = _space(workspace, lambda: gdn_paged_prefill_workspace_bytes(
        H, kv, d, code, n, T), q, stream, dev)
    _run("gdn_paged_prefill", dev, stream, gdn_paged_dims_t(H, kv, d, code, scale),
         _arg("q", q, (T, H, d), dt, dev), _arg("k_cache", k_cache, (n_blocks, kv, bs, d), dt, dev),
         _arg("v_cache", v_cache, (n_blocks, kv, bs, d), dt, dev), n_blocks, bs,
         _table_arg(block_table, n, dev), block_table.shape[1],
         _arg("cu_seqlens", cu_seqlens, (n + 1,), _I32, dev),
         _arg("seq_lens", seq_lens, (n,), _I32, dev), n, T, _arg("o", o, (T, H, d), dt, dev), ws,
         ws_bytes)
    return o


def _latent_dims(H, rank, d_rope, d_nope, d_v, scale):
    return gdn_latent_dims_t(H, rank, d_rope, d_nope, d_v, GDN_DTYPE_BF16, scale)


def gdn_latent_decode_workspace_bytes(H, rank, d_rope, d_nope, d_v, batch, n_pos=1):
    dims = _latent_dims(int(H), int(rank), int(d_rope), int(d_nope), int(d_v), 1.0)
    out = _SZ(0)
    _check("gdn_latent_decode_workspace_bytes", lib().gdn_latent_decode_workspace_bytes(
        ctypes.byref(dims), int(batch), int(n_pos), ctypes.byref(out)))
    return int(out.value)


def gdn_latent_decode(q_nope, q_pe, w_kv, cache, block_table, seq_lens, scale=1.0, o=None,
                      workspace=None, stream=None):
    """Latent attention of the newest tokens, absorbed form (bf16). q_nope [B, H, d] or
    [B, P, H, d], q_pe likewise with d_rope; w_kv [H, d_nope + d_v, rank] (the rows of the key
    up projection, then of the value's; d_nope == d_v); cache [n_blocks, block_size, rank +
    d_rope]; block_table [B, max_blocks] int32; seq_lens [B] int32. Returns o, shaped as
    q_nope."""
    shape = q_nope.shape
    if len(shape) == 3:  # one position per request
        (B, H, dn), P = shape, 1
    else:
        B, P, H, dn = shape
    rank, rope = w_kv.shape[2], q_pe.shape[-1]
    dv = w_kv.shape[1] - dn
    n_blocks, bs, _ = cache.shape
    dev = _gpu(q_nope)
    o_shape = (*shape[:-1], dv)
    o = _new(o_shape, _BF16, q_nope, stream) if o is None else o
    ws, ws_bytes = _space(workspace, lambda: gdn_latent_decode_workspace_bytes(
        H, rank, rope, dn, dv, B, P), q_nope, stream, dev)
    _run("gdn_latent_decode", dev, stream, _latent_dims(H, rank, rope, dn, dv, scale),
         _arg("q_nope", q_nope, shape, _BF16, dev),
         _arg("q_pe", q_pe, (*shape[:-1], rope), _BF16, dev),
         _arg("w_kv", w_kv, (H, dn + dv, rank), _BF16, dev),
         _arg("cache", cache, (n_blocks, bs, rank + rope), _BF16, dev), n_blocks, bs,
         _table_arg(block_table, B, dev), block_table.shape[1],
         _arg("seq_lens", seq_lens, (B,), _I32, dev), B, P, _arg("o", o, o_shape, _BF16, dev), ws,
         ws_bytes)
    return o


def gdn_latent_prefill_workspace_bytes(H, rank, d_rope, d_nope, d_v, n_seqs, total_tokens,
                                       total_keys):
    dims = _latent_dims(int(H), int(rank), int(d_rope), int(d_nope), int(d_v), 1.0)
    out = _SZ(0)
    _check("gdn_latent_prefill_workspace_bytes", lib().gdn_latent_prefill_workspace_bytes(
        ctypes.byref(dims), int(n_seqs), int(total_tokens), int(total_keys), ctypes.byref(out)))
    return int(out.value)


def gdn_latent_prefill(q_nope, q_pe, w_kv, cache, block_table, cu_seqlens, seq_lens, total_keys,
                       scale=1.0, o=None, workspace=None, stream=None):
    """Latent attention of packed new tokens, expanded form, causal (bf16). q_nope [T, H, d],
    q_pe [T, H, d_rope]; w_kv, cache and block_table as gdn_latent_decode; cu_seqlens [n + 1]
    int32; seq_lens [n] int32, the new tokens included; total_keys >= the sum of seq_lens.
    Returns o [T, H, d]."""
    T, H, dn = q_nope.shape
    n = seq_lens.numel()
    rank, rope = w_kv.shape[2], q_pe.shape[2]
    dv = w_kv.shape[1] - dn
    n_blocks, bs, _ = cache.shape
    dev = _gpu(q_nope)
    o = _new((T, H, dv), _BF16, q_nope, stream) if o is None else o
    ws, ws_bytes = _space(workspace, lambda: gdn_latent_prefill_workspace_bytes(
        H, rank, rope, dn, dv, n, T, total_keys), q_nope, stream, dev)
    _run("gdn_latent_prefill", dev, stream, _latent_dims(H, rank, rope, dn, dv, scale),
         _arg("q_nope", q_nope, (T, H, dn), _BF16, dev),
         _arg("q_pe", q_pe, (T, H, rope), _BF16, dev),
         _arg("w_kv", w_kv, (H, dn + dv, rank), _BF16, dev),
         _arg("cache", cache, (n_blocks, bs, rank + rope), _BF16, dev), n_blocks, bs,
         _table_arg(block_table, n, dev), block_table.shape[1],
         _arg("cu_seqlens", cu_seqlens, (n + 1,), _I32, dev),
         _arg("seq_lens", seq_lens, (n,), _I32, dev), n, T, int(total_keys),
         _arg("o", o, (T, H, dv), _BF16, dev), ws, ws_bytes)
    return o
