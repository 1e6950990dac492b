"""Python binding of libgdn.so, the MI355X Gated DeltaNet engine.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in ``include/gdn.h``.  Torch supplies device
memory and the current HIP stream.  There is no fallback: if the library is
missing or fails to load, importing the entry points raises.

Entry points (same names as the C ABI):

``gdn_prefill_chunked``       chunked prefill with explicit initial/final state
``gdn_recurrent_step``        token-by-token step with compact state-update capture
``gdn_replay_state_updates``  replay of captured (decay, key, delta) records
``gdn_state_snapshot``        immutable copy of a state set
``gdn_prefill_workspace_bytes``
``gdn_linear_prefill``        linear attention with a decay for each head, whole sequences
``gdn_linear_step``           the same token by token, with capture
``gdn_verify_drafts``         drafted tokens against the target's probabilities
``gdn_block_norm``            norms around a block, fused with gate, residual and scale
``gdn_cache_append``          new keys (rotated) and values into a paged cache
``gdn_cache_attention``       attention of new tokens over the paged cache
``gdn_cache_copy_pages``      pages copied inside the cache
``gdn_beam_select``           the best continuations of a beam search
``gdn_state_reorder``         states moved from each parent to its beam
"""

from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_F32, GDN_F16, GDN_BF16 = 0, 1, 2
GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_HIP = 0, 1, 2, 3
_DTYPES = {torch.float32: GDN_F32, torch.float16: GDN_F16, torch.bfloat16: GDN_BF16}
EXPORTED = ("gdn_abi_version", "gdn_prefill_workspace_bytes", "gdn_prefill_chunked",
            "gdn_prefill_chunked_states", "gdn_prefill_chunked_ex", "gdn_recurrent_step",
            "gdn_recurrent_step_ex", "gdn_replay_state_updates", "gdn_state_snapshot",
            "gdn_status_string", "gdn_last_error", "gdn_profile_enable", "gdn_profile_collect",
            "gdn_prefill_chunked_noalloc", "gdn_linear_workspace_bytes", "gdn_linear_prefill", "gdn_linear_step",
            "gdn_verify_workspace_bytes", "gdn_verify_drafts", "gdn_block_norm", "gdn_cache_append",
            "gdn_cache_attention_workspace_bytes", "gdn_cache_attention", "gdn_beam_workspace_bytes",
            "gdn_beam_select", "gdn_state_reorder")
GDN_NOALLOC_SCRATCH_BYTES = 128 * 1024 * 1024


class gdn_prologue(ctypes.Structure):
    _fields_ = [("qk_l2norm", ctypes.c_int32), ("qk_l2norm_eps", ctypes.c_float),
                ("beta_is_logit", ctypes.c_int32), ("gate_A_log", ctypes.c_void_p),
                ("gate_dt_bias", ctypes.c_void_p)]


class Prologue:
    """Input prologue of the *_ex calls: qk_l2norm (with eps), beta given as
    logits, and the gate -exp(A_log[h]) * softplus(g + dt_bias[h]) when A_log
    (fp32 [Hv] on the device) is set.  Tensors are kept alive by this object."""

    def __init__(self, qk_l2norm=False, eps=1e-6, beta_is_logit=False, A_log=None, dt_bias=None):
        self.qk_l2norm, self.eps, self.beta_is_logit = bool(qk_l2norm), float(eps), bool(beta_is_logit)
        self.A_log, self.dt_bias = A_log, dt_bias

    def as_c(self, device):
        for t, n in ((self.A_log, "A_log"), (self.dt_bias, "dt_bias")):
            _need(t, n, torch.float32, device)
        return gdn_prologue(int(self.qk_l2norm), self.eps, int(self.beta_is_logit),
                            None if self.A_log is None else self.A_log.data_ptr(),
                            None if self.dt_bias is None else self.dt_bias.data_ptr())


class gdn_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("Hv", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class gdn_verify_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("target_row_stride", ctypes.c_int64), ("draft_row_stride", ctypes.c_int64)]


class gdn_norm_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("D", ctypes.c_int32), ("group", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate_act", ctypes.c_int32), ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)]


class gdn_cache_shape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class gdn_append_shape(ctypes.Structure):
    _fields_ = [("q_token_stride", ctypes.c_int64), ("k_token_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("rotary", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("axes", ctypes.c_int32)]


class gdn_beam_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("W", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("eos_token", ctypes.c_int32), ("pad_token", ctypes.c_int32),
                ("row_stride", ctypes.c_int64)]


class gdn_reorder_shape(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int64), ("src_layer_stride", ctypes.c_int64), ("dst_layer_stride", ctypes.c_int64),
                ("src_rows", ctypes.c_int64), ("dst_rows", ctypes.c_int64), ("row_bytes", ctypes.c_int64),
                ("src_group", ctypes.c_int64), ("G", ctypes.c_int32), ("W", ctypes.c_int32)]


class GdnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgdn.so (once).  Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m gated_deltanet_03_amd._build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    shp = ctypes.POINTER(gdn_shape)
    lib.gdn_abi_version.restype = i32
    lib.gdn_abi_version.argtypes = []
    lib.gdn_prefill_workspace_bytes.restype = sz
    lib.gdn_prefill_workspace_bytes.argtypes = [shp, i32, i32]
    lib.gdn_prefill_chunked.restype = i32
    lib.gdn_prefill_chunked.argtypes = [shp, vp, vp, vp, vp, vp, vp, i64, vp, i32, vp, vp, vp, sz, vp]
    lib.gdn_prefill_chunked_noalloc.restype = i32
    lib.gdn_prefill_chunked_noalloc.argtypes = [shp, vp, vp, vp, vp, vp, vp, i64, vp, i32, vp, vp, vp]
    lib.gdn_recurrent_step.restype = i32
    lib.gdn_prefill_chunked_states.argtypes = [shp, vp, vp, vp, vp, vp, vp, i64, vp, i32, vp, vp, vp, i64, vp,
                                               sz, vp]
    lib.gdn_prefill_chunked_states.restype = i32
    pro = ctypes.POINTER(gdn_prologue)
    lib.gdn_prefill_chunked_ex.argtypes = [shp, pro, vp, vp, vp, vp, vp, vp, i64, vp, i32, vp, vp, vp, i64, vp,
                                           sz, vp]
    lib.gdn_prefill_chunked_ex.restype = i32
    lib.gdn_recurrent_step_ex.argtypes = [shp, pro, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, i32, vp, i32, vp, vp]
    lib.gdn_recurrent_step_ex.restype = i32
    lib.gdn_recurrent_step.argtypes = [shp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, i32, vp, i32, vp, vp]
    lib.gdn_replay_state_updates.restype = i32
    lib.gdn_replay_state_updates.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, vp, vp]
    lib.gdn_state_snapshot.restype = i32
    lib.gdn_state_snapshot.argtypes = [vp, vp, i64, i32, i32, i32, vp]
    lib.gdn_linear_workspace_bytes.restype = sz
    lib.gdn_linear_workspace_bytes.argtypes = [shp, i32]
    lib.gdn_linear_prefill.restype = i32
    lib.gdn_linear_prefill.argtypes = [shp, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp, vp, sz, vp]
    lib.gdn_linear_step.restype = i32
    lib.gdn_linear_step.argtypes = [shp, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp, i32, vp, vp, vp]
    vshp, nshp = ctypes.POINTER(gdn_verify_shape), ctypes.POINTER(gdn_norm_shape)
    lib.gdn_verify_workspace_bytes.restype = sz
    lib.gdn_verify_workspace_bytes.argtypes = [vshp]
    lib.gdn_verify_drafts.restype = i32
    lib.gdn_verify_drafts.argtypes = [vshp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdn_block_norm.restype = i32
    lib.gdn_block_norm.argtypes = [nshp, vp, vp, vp, vp, vp, vp, vp, vp]
    cshp, ashp = ctypes.POINTER(gdn_cache_shape), ctypes.POINTER(gdn_append_shape)
    bshp, rshp = ctypes.POINTER(gdn_beam_shape), ctypes.POINTER(gdn_reorder_shape)
    lib.gdn_cache_append.restype = i32
    lib.gdn_cache_append.argtypes = [cshp, ashp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.gdn_cache_attention_workspace_bytes.restype = sz
    lib.gdn_cache_attention_workspace_bytes.argtypes = [cshp, i32]
    lib.gdn_cache_attention.restype = i32
    lib.gdn_cache_attention.argtypes = [cshp, vp, i64, vp, vp, vp, vp, vp, ctypes.c_float, i32, vp, vp, sz, vp]
    lib.gdn_beam_workspace_bytes.restype = sz
    lib.gdn_beam_workspace_bytes.argtypes = [bshp]
    lib.gdn_beam_select.restype = i32
    lib.gdn_beam_select.argtypes = [bshp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdn_state_reorder.restype = i32
    lib.gdn_state_reorder.argtypes = [rshp, vp, vp, vp, vp, vp]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [i32]
    lib.gdn_last_error.restype = ctypes.c_char_p
    lib.gdn_last_error.argtypes = []
    lib.gdn_profile_enable.restype = i32
    lib.gdn_profile_enable.argtypes = [i32]
    lib.gdn_profile_collect.restype = i32
    lib.gdn_profile_collect.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_int32), i32]
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != GDN_OK:
        lib = load_library()
        raise GdnError(status, f"{lib.gdn_status_string(status).decode()}: {lib.gdn_last_error().decode()}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    if device is None or device.type != "cuda":
        return ctypes.c_void_p(0)
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtype=None, device=None):
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _expect(t, name, numel, at_least=False):
    """Raise ValueError unless tensor t holds exactly (or at least) numel elements.
    The C ABI sees bare pointers, so sizes are checked here, before any call."""
    if t is None:
        return
    n = t.numel()
    if (n < numel) if at_least else (n != numel):
        rel = "at least " if at_least else ""
        raise ValueError(f"{name} has {n} elements, expected {rel}{numel}")


def _check_tokens(sh, q, k, v, g, beta, o, cu_seqlens):
    """Token tensors against the problem description built from q and v."""
    ntok = sh.T if cu_seqlens is not None else sh.B * sh.T
    if tuple(k.shape) != tuple(q.shape):
        raise ValueError(f"k has shape {tuple(k.shape)}, q has {tuple(q.shape)}")
    if v.dim() != q.dim() or tuple(v.shape[:-2]) != tuple(q.shape[:-2]):
        raise ValueError(f"v has shape {tuple(v.shape)}; its leading dims must match q's {tuple(q.shape[:-2])}")
    _expect(v, "v", ntok * sh.Hv * sh.dv)
    for t, n in ((g, "g"), (beta, "beta")):
        if tuple(t.shape) != tuple(v.shape[:-1]):
            raise ValueError(f"{n} has shape {tuple(t.shape)}, expected {tuple(v.shape[:-1])}")
    if o is not None and tuple(o.shape) != tuple(v.shape):
        raise ValueError(f"o has shape {tuple(o.shape)}, expected {tuple(v.shape)}")
    if cu_seqlens is not None and cu_seqlens.dim() != 1:
        raise ValueError("cu_seqlens must be 1-D [N+1]")


def _check_states(sh, initial_state, stride, final_state):
    """initial_state covers (B-1)*stride + Hv*dk*dv elements; final_state is [B, Hv, dk, dv]."""
    per = sh.Hv * sh.dk * sh.dv
    if stride < 0:
        raise ValueError(f"initial_state_batch_stride={stride} < 0")
    if initial_state is not None and sh.B > 0:
        _expect(initial_state, "initial_state", (sh.B - 1) * stride + per, at_least=True)
    if final_state is not None and tuple(final_state.shape) != (sh.B, sh.Hv, sh.dk, sh.dv):
        raise ValueError(f"final_state has shape {tuple(final_state.shape)}, expected "
                         f"{(sh.B, sh.Hv, sh.dk, sh.dv)}")


def _shape_from(q, k, v, scale, cu_seqlens):
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError("dense q must be [B, T, Hq, dk]")
        B, T, Hq, dk = q.shape
    else:
        if q.dim() == 4:
            if q.shape[0] != 1:
                raise ValueError("ragged q must be [1, T, Hq, dk] or [T, Hq, dk]")
            q = q[0]
        T, Hq, dk = q.shape
        B = cu_seqlens.numel() - 1
    Hv, dv = v.shape[-2], v.shape[-1]
    if q.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if scale is None:
        scale = dk ** -0.5
    return gdn_shape(B, T, Hq, Hv, dk, dv, float(scale), _DTYPES[q.dtype])


def gdn_prefill_workspace_bytes(shape: gdn_shape, chunk_size: int, ragged: bool) -> int:
    return int(load_library().gdn_prefill_workspace_bytes(ctypes.byref(shape), chunk_size, int(bool(ragged))))


def gdn_prefill_chunked(q, k, v, g, beta, *, scale=None, initial_state=None,
                        initial_state_batch_stride=None, cu_seqlens=None, chunk_size=64,
                        o=None, final_state=None, output_final_state=True, workspace=None):
    """Chunked prefill.  Dense q/k [B,T,Hq,dk], v [B,T,Hv,dv], g/beta [B,T,Hv];
    ragged: the same without B (or B=1) plus cu_seqlens int32 [N+1] on the device.
    Returns (o, final_state or None)."""
    return _prefill(q, k, v, g, beta, scale, initial_state, initial_state_batch_stride, cu_seqlens,
                    chunk_size, o, final_state, output_final_state, workspace, False, None, None)[:2]


def gdn_prefill_chunked_noalloc(q, k, v, g, beta, *, scale=None, initial_state=None,
                                initial_state_batch_stride=None, cu_seqlens=None, chunk_size=64,
                                o=None, final_state=None, output_final_state=True):
    """gdn_prefill_chunked with the library's fixed device scratch array as the
    workspace (the C entry point allocates nothing; pass ``o`` and
    ``final_state`` to allocate nothing here either).  Returns (o, final_state
    or None)."""
    lib = load_library()
    dev = q.device
    sh = _shape_from(q, k, v, scale, cu_seqlens)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    _need(initial_state, "initial_state", torch.float32, dev)
    if o is None:
        o = torch.empty(v.shape, dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, dev)
    per = sh.Hv * sh.dk * sh.dv
    if final_state is None and output_final_state:
        final_state = torch.empty((sh.B, sh.Hv, sh.dk, sh.dv), dtype=torch.float32, device=dev)
    _need(final_state, "final_state", torch.float32, dev)
    if initial_state_batch_stride is None:
        initial_state_batch_stride = 0 if (initial_state is not None and initial_state.shape[0] == 1
                                           and sh.B > 1) else per
    _check_tokens(sh, q, k, v, g, beta, o, cu_seqlens)
    _check_states(sh, initial_state, int(initial_state_batch_stride), final_state)
    _check(lib.gdn_prefill_chunked_noalloc(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                           _ptr(initial_state), int(initial_state_batch_stride),
                                           _ptr(cu_seqlens), int(chunk_size), _ptr(o), _ptr(final_state),
                                           _stream(dev)))
    return o, final_state


def gdn_prefill_chunked_states(q, k, v, g, beta, *, scale=None, initial_state=None,
                               initial_state_batch_stride=None, cu_seqlens=None, chunk_size=64,
                               o=None, final_state=None, output_final_state=True, workspace=None,
                               chunk_states=None, num_chunks=None):
    """Chunked prefill that also returns the state after every chunk:
    chunk_states [sum_s ceil(L_s / chunk_size), Hv, dk, dv] fp32, sequence s's
    chunk j at index sum_{s'<s} ceil(L_s'/chunk_size) + j.  Without
    ``chunk_states`` or ``num_chunks`` the count is taken from the lengths
    (ragged input: one device-to-host read of cu_seqlens).
    Returns (o, final_state or None, chunk_states)."""
    return _prefill(q, k, v, g, beta, scale, initial_state, initial_state_batch_stride, cu_seqlens,
                    chunk_size, o, final_state, output_final_state, workspace, True, chunk_states, num_chunks)


def gdn_prefill_chunked_ex(q, k, v, g, beta, *, prologue=None, scale=None, initial_state=None,
                           initial_state_batch_stride=None, cu_seqlens=None, chunk_size=64, o=None,
                           final_state=None, output_final_state=True, workspace=None, chunk_states=None,
                           num_chunks=None, emit_chunk_states=False):
    """Chunked prefill with the input prologue (a ``Prologue`` or None) and,
    with ``emit_chunk_states`` (or a ``chunk_states`` buffer), the boundary
    states.  Returns (o, final_state or None, chunk_states or None)."""
    emit = emit_chunk_states or chunk_states is not None or num_chunks is not None
    return _prefill(q, k, v, g, beta, scale, initial_state, initial_state_batch_stride, cu_seqlens,
                    chunk_size, o, final_state, output_final_state, workspace, emit, chunk_states, num_chunks,
                    prologue=prologue if prologue is not None else Prologue())


def _prefill(q, k, v, g, beta, scale, initial_state, initial_state_batch_stride, cu_seqlens, chunk_size,
             o, final_state, output_final_state, workspace, emit, chunk_states, num_chunks, prologue=None):
    lib = load_library()
    dev = q.device
    sh = _shape_from(q, k, v, scale, cu_seqlens)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    _need(initial_state, "initial_state", torch.float32, dev)
    if o is None:
        o = torch.empty(v.shape, dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, dev)
    per = sh.Hv * sh.dk * sh.dv
    if final_state is None and output_final_state:
        final_state = torch.empty((sh.B, sh.Hv, sh.dk, sh.dv), dtype=torch.float32, device=dev)
    _need(final_state, "final_state", torch.float32, dev)
    if initial_state_batch_stride is None:
        initial_state_batch_stride = 0 if (initial_state is not None and initial_state.shape[0] == 1
                                           and sh.B > 1) else per
    _check_tokens(sh, q, k, v, g, beta, o, cu_seqlens)
    _check_states(sh, initial_state, int(initial_state_batch_stride), final_state)
    need = gdn_prefill_workspace_bytes(sh, chunk_size, cu_seqlens is not None)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", None, dev)
    common = (ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
              int(initial_state_batch_stride), _ptr(cu_seqlens), int(chunk_size), _ptr(o), _ptr(final_state))
    if prologue is not None:
        pc = prologue.as_c(dev)
        buf = None
        if emit:
            chunk_states, buf = _chunk_buffer(sh, cu_seqlens, chunk_size, chunk_states, num_chunks, dev)
        ncs = 0 if buf is None else int(chunk_states.numel() // max(per, 1))
        _check(lib.gdn_prefill_chunked_ex(common[0], ctypes.byref(pc), *common[1:], _ptr(buf), ncs,
                                          _ptr(workspace), workspace.numel(), _stream(dev)))
        return o, final_state, chunk_states if emit else None
    if not emit:
        _check(lib.gdn_prefill_chunked(*common, _ptr(workspace), workspace.numel(), _stream(dev)))
        return o, final_state, None
    chunk_states, buf = _chunk_buffer(sh, cu_seqlens, chunk_size, chunk_states, num_chunks, dev)
    _check(lib.gdn_prefill_chunked_states(*common, _ptr(buf), int(chunk_states.numel() // max(per, 1)),
                                          _ptr(workspace), workspace.numel(), _stream(dev)))
    return o, final_state, chunk_states


def _chunk_buffer(sh, cu_seqlens, chunk_size, chunk_states, num_chunks, dev):
    """(chunk_states view, buffer with an address) for the boundary states."""
    if chunk_states is not None:
        _need(chunk_states, "chunk_states", torch.float32, dev)
        if chunk_states.dim() != 4 or tuple(chunk_states.shape[1:]) != (sh.Hv, sh.dk, sh.dv):
            raise ValueError(f"chunk_states has shape {tuple(chunk_states.shape)}, expected "
                             f"[num_chunks, {sh.Hv}, {sh.dk}, {sh.dv}]")
        return chunk_states, chunk_states
    if num_chunks is None:
        if cu_seqlens is None:
            num_chunks = sh.B * (-(-sh.T // chunk_size))
        else:
            lens = cu_seqlens.cpu().diff()
            num_chunks = int(((lens + chunk_size - 1) // chunk_size).sum())
    # at least one entry, so the buffer has an address even with no chunks
    buf = torch.empty((max(int(num_chunks), 1), sh.Hv, sh.dk, sh.dv), dtype=torch.float32, device=dev)
    return buf[:int(num_chunks)], buf


def gdn_recurrent_step_ex(q, k, v, g, beta, *, prologue=None, **kw):
    """Recurrent step with the input prologue (a ``Prologue`` or None); the
    other arguments as gdn_recurrent_step.  Returns (o, final_state, state_update)."""
    return gdn_recurrent_step(q, k, v, g, beta, _prologue=prologue if prologue is not None else Prologue(), **kw)


def gdn_recurrent_step(q, k, v, g, beta, *, scale=None, initial_state=None,
                       initial_state_batch_stride=None, cu_seqlens=None, o=None, final_state=None,
                       output_final_state=True, state_update_capacity=0, capture_count=None,
                       state_update_active=1, state_update=None, _prologue=None):
    """Recurrent step with optional compact capture.  Returns (o, final_state, state_update)."""
    lib = load_library()
    dev = q.device
    sh = _shape_from(q, k, v, scale, cu_seqlens)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, dev)
    _need(g, "g", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    _need(initial_state, "initial_state", torch.float32, dev)
    _need(capture_count, "capture_count", torch.int32, dev)
    if o is None:
        o = torch.empty(v.shape, dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, dev)
    per = sh.Hv * sh.dk * sh.dv
    if final_state is None and output_final_state:
        final_state = torch.empty((sh.B, sh.Hv, sh.dk, sh.dv), dtype=torch.float32, device=dev)
    _need(final_state, "final_state", torch.float32, dev)
    if initial_state_batch_stride is None:
        initial_state_batch_stride = 0 if (initial_state is not None and initial_state.shape[0] == 1
                                           and sh.B > 1) else per
    cap = int(state_update_capacity)
    if cap > 0 and state_update is None:
        R = sh.Hv + sh.Hq * sh.dk + sh.Hv * sh.dv
        state_update = torch.empty((sh.B, cap, R), dtype=torch.float32, device=dev)
    _need(state_update, "state_update", torch.float32, dev)
    _check_tokens(sh, q, k, v, g, beta, o, cu_seqlens)
    _check_states(sh, initial_state, int(initial_state_batch_stride), final_state)
    if cap < 0:
        raise ValueError(f"state_update_capacity={cap} < 0")
    if cap > 0:
        if capture_count is None:
            raise ValueError("capture_count is required when state_update_capacity > 0")
        _expect(capture_count, "capture_count", sh.B, at_least=True)
        R = sh.Hv + sh.Hq * sh.dk + sh.Hv * sh.dv
        _expect(state_update, "state_update", sh.B * cap * R, at_least=True)
    rest = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), int(initial_state_batch_stride),
            _ptr(cu_seqlens), _ptr(o), _ptr(final_state), cap, _ptr(capture_count), int(state_update_active),
            _ptr(state_update), _stream(dev))
    if _prologue is None:
        _check(lib.gdn_recurrent_step(ctypes.byref(sh), *rest))
    else:
        pc = _prologue.as_c(dev)
        _check(lib.gdn_recurrent_step_ex(ctypes.byref(sh), ctypes.byref(pc), *rest))
    return o, final_state, state_update


def gdn_replay_state_updates(state, state_update, replay_count, *, Hq, state_update_capacity=None):
    """Replay the first replay_count[b] records of each row onto state (in place)."""
    lib = load_library()
    dev = state.device
    B, Hv, dk, dv = state.shape
    cap = state_update.shape[1] if state_update_capacity is None else int(state_update_capacity)
    _need(state, "state", torch.float32, dev)
    _need(state_update, "state_update", torch.float32, dev)
    _need(replay_count, "replay_count", torch.int32, dev)
    if state.dim() != 4:
        raise ValueError(f"state must be [B, Hv, dk, dv], got shape {tuple(state.shape)}")
    Hq = int(Hq)
    if Hq <= 0 or Hv % Hq != 0:
        raise ValueError(f"Hq={Hq} must be positive and divide Hv={Hv}")
    if cap < 0:
        raise ValueError(f"state_update_capacity={cap} < 0")
    R = Hv + Hq * dk + Hv * dv
    if state_update.dim() == 3 and state_update.shape[-1] != R:
        raise ValueError(f"state_update records hold {state_update.shape[-1]} floats; Hv + Hq*dk + Hv*dv = {R}")
    if cap > 0:
        _expect(state_update, "state_update", B * cap * R, at_least=True)
        _expect(replay_count, "replay_count", B, at_least=True)
    _check(lib.gdn_replay_state_updates(B, int(Hq), Hv, dk, dv, cap, _ptr(state_update), _ptr(replay_count),
                                        _ptr(state), _stream(dev)))
    return state


def gdn_state_snapshot(src, dst=None):
    """Bitwise copy of a [N, Hv, dk, dv] fp32 state set, ordered on the current stream."""
    lib = load_library()
    dev = src.device
    _need(src, "src", torch.float32, dev)
    if dst is None:
        dst = torch.empty_like(src)
    _need(dst, "dst", torch.float32, dev)
    if src.dim() != 4:
        raise ValueError(f"src must be [N, Hv, dk, dv], got shape {tuple(src.shape)}")
    if tuple(dst.shape) != tuple(src.shape):
        raise ValueError(f"dst has shape {tuple(dst.shape)}, src {tuple(src.shape)}")
    N, Hv, dk, dv = src.shape
    _check(lib.gdn_state_snapshot(_ptr(src), _ptr(dst), N, Hv, dk, dv, _stream(dev)))
    return dst


# ---------------------------------------------------------------------------
# Linear attention with a decay for each head, draft verification, block norms
# ---------------------------------------------------------------------------
def _addr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it (1.0 us less a call);
# torch keeps that query to itself, so the public one stands in where it is missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on_gpu(dev):
    """The library reads device memory only; a host pointer would fault the GPU."""
    if dev.type != "cuda":
        raise ValueError(f"tensors are on {dev}, expected a GPU")
    return _raw_stream(dev.index)


_kept = {}


def _descriptor(cls, key):
    """The C struct of these values and a reference to it.  A serving loop makes the
    same few descriptors over and over; they are kept by value."""
    hit = _kept.get((cls, key))
    if hit is None:
        for (name, kind), x in zip(cls._fields_, key):
            if kind is ctypes.c_int32 and x >= 1 << 31:   # ctypes would keep its low bits
                raise ValueError(f"{name}={x} does not fit 32 bits")
        if len(_kept) >= 1024:
            _kept.clear()
        sh = cls(*key)
        hit = _kept[cls, key] = (sh, ctypes.byref(sh))
    return hit


def _scratch(need, dev):
    return torch.empty(need, dtype=torch.uint8, device=dev) if 0 < need < 1 << 62 else None


def _linear_common(q, k, v, g, scale, initial_state, stride, cu_seqlens, o, final_state, output_final_state):
    """Checks shared by gdn_linear_prefill and gdn_linear_step."""
    dev, dtype, qs, vs = q.device, q.dtype, q.shape, v.shape
    if cu_seqlens is None:
        if len(qs) != 4:
            raise ValueError("dense q must be [B, T, Hq, dk]")
        B, T, Hq, dk = qs
    else:
        if len(qs) == 4 and qs[0] != 1:
            raise ValueError("ragged q must be [1, T, Hq, dk] or [T, Hq, dk]")
        T, Hq, dk = qs[-3:]
        B = cu_seqlens.shape[0] - 1 if cu_seqlens.dim() == 1 else -1
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if B < 0:
            raise ValueError("cu_seqlens must be 1-D [N+1]")
    Hv, dv = vs[-2:]
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    _need(q, "q")
    _need(k, "k", dtype, dev)
    _need(v, "v", dtype, dev)
    _need(g, "g", torch.float32, dev)
    if Hq <= 0 or Hv % Hq != 0:
        raise ValueError(f"Hv={Hv} must be a multiple of Hq={Hq}")
    if k.shape != qs:
        raise ValueError(f"k has shape {tuple(k.shape)}, q has {tuple(qs)}")
    if len(vs) != len(qs) or vs[:-2] != qs[:-2]:
        raise ValueError(f"v has shape {tuple(vs)}; its leading dims must match q's {tuple(qs[:-2])}")
    g_stride = 0 if g.dim() == 1 else Hv
    if g.shape != ((Hv,) if g_stride == 0 else vs[:-1]):
        raise ValueError(f"g has shape {tuple(g.shape)}, expected {(Hv,)} or {tuple(vs[:-1])}")
    if o is None:
        o = torch.empty_like(v)
    else:
        _need(o, "o", dtype, dev)
        if o.shape != vs:
            raise ValueError(f"o has shape {tuple(o.shape)}, expected {tuple(vs)}")
    per, states = Hv * dk * dv, (B, Hv, dk, dv)
    same = False
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, dev)
        same = initial_state.shape == states
        if stride is None:
            stride = 0 if B > 1 and initial_state.shape[0] == 1 else per
        stride = int(stride)
        if stride < 0:
            raise ValueError(f"initial_state_batch_stride={stride} < 0")
        if B > 0 and not (same and stride <= per):
            _expect(initial_state, "initial_state", (B - 1) * stride + per, at_least=True)
    else:
        stride = per
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, dev)
        if final_state.shape != states:
            raise ValueError(f"final_state has shape {tuple(final_state.shape)}, expected {states}")
    elif output_final_state:
        final_state = torch.empty_like(initial_state) if same else torch.empty(states, dtype=torch.float32, device=dev)
    sh, ref = _descriptor(gdn_shape, (B, T, Hq, Hv, dk, dv, dk ** -0.5 if scale is None else float(scale), code))
    return sh, ref, g_stride, stride, o, final_state


def gdn_linear_workspace_bytes(shape: gdn_shape, ragged: bool) -> int:
    """Bytes gdn_linear_prefill needs for this shape (0: none)."""
    n = load_library().gdn_linear_workspace_bytes(ctypes.byref(shape), int(bool(ragged)))
    if n == ctypes.c_size_t(-1).value:
        _check(GDN_ERR_INVALID_ARG)
    return int(n)


def gdn_linear_prefill(q, k, v, g, *, scale=None, initial_state=None, initial_state_batch_stride=None,
                       cu_seqlens=None, o=None, final_state=None, output_final_state=True, workspace=None):
    """Linear attention with a decay for each head over whole sequences:
    S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, g <= 0.

    Dense q/k [B,T,Hq,dk], v [B,T,Hv,dv]; ragged: the same without B (or B=1)
    plus cu_seqlens int32 [N+1].  g fp32: log decays [..., Hv] per token, or [Hv]
    the same at every token.  Returns (o, final_state or None)."""
    lib = load_library()
    sh, ref, g_stride, stride, o, final_state = _linear_common(
        q, k, v, g, scale, initial_state, initial_state_batch_stride, cu_seqlens, o, final_state, output_final_state)
    dev = q.device
    stream = _on_gpu(dev)
    if workspace is None:   # an invalid shape is named by the call itself
        workspace = _scratch(lib.gdn_linear_workspace_bytes(ref, cu_seqlens is not None), dev)
    else:
        _need(workspace, "workspace", None, dev)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.gdn_linear_prefill(ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), g_stride,
                                _addr(initial_state), stride, _addr(cu_seqlens), o.data_ptr(), _addr(final_state),
                                _addr(workspace), nbytes, stream)
    if st:
        _check(st)
    return o, final_state


def gdn_linear_step(q, k, v, g, *, scale=None, initial_state=None, initial_state_batch_stride=None, cu_seqlens=None,
                    o=None, final_state=None, output_final_state=True, state_update_capacity=0, capture_count=None,
                    state_update=None):
    """gdn_linear_prefill's recurrence token by token (for a few tokens a row),
    with g of any sign and optional capture of (decay, key, value) records that
    gdn_replay_state_updates applies.  Returns (o, final_state or None,
    state_update or None)."""
    lib = load_library()
    sh, ref, g_stride, stride, o, final_state = _linear_common(
        q, k, v, g, scale, initial_state, initial_state_batch_stride, cu_seqlens, o, final_state, output_final_state)
    dev = q.device
    cap = int(state_update_capacity)
    if cap > 0:
        if capture_count is None:
            raise ValueError("capture_count is required when state_update_capacity > 0")
        R = sh.Hv + sh.Hq * sh.dk + sh.Hv * sh.dv
        if state_update is None:
            state_update = torch.empty((sh.B, cap, R), dtype=torch.float32, device=dev)
        _need(state_update, "state_update", torch.float32, dev)
        _need(capture_count, "capture_count", torch.int32, dev)
        _expect(capture_count, "capture_count", sh.B, at_least=True)
        _expect(state_update, "state_update", sh.B * cap * R, at_least=True)
    stream = _on_gpu(dev)
    st = lib.gdn_linear_step(ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), g_stride,
                             _addr(initial_state), stride, _addr(cu_seqlens), o.data_ptr(), _addr(final_state), cap,
                             _addr(capture_count), _addr(state_update), stream)
    if st:
        _check(st)
    return o, final_state, state_update


def _rows3(t, name, B, n, V, dtype, dev):
    """Elements between the rows of a [B, n, V] tensor whose rows are evenly spaced."""
    if t.shape != (B, n, V):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(B, n, V)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.is_contiguous():
        return V
    s0, s1, s2 = t.stride()
    if V > 1 and s2 != 1:
        raise ValueError(f"{name} must be contiguous along the vocabulary")
    row = s1 if n > 1 else (s0 if B > 1 else V)
    if row < V or (B > 1 and s0 != n * row):
        raise ValueError(f"{name} must have evenly spaced rows, got strides {t.stride()}")
    return row


def gdn_verify_drafts(target_probs, draft_probs, draft_tokens, uniforms, *, draft_count=None, tokens=None,
                      emit_count=None, workspace=None):
    """Verify drafted tokens against the target's probabilities.

    target_probs [B, K+1, V], draft_probs [B, K, V] of the same dtype (None:
    deterministic drafts), draft_tokens int32 [B, K], uniforms fp32 [B, K+1] in
    [0, 1), draft_count int32 [B] (None: K each; negative: idle row).  Rows of
    the probabilities may be padded (evenly spaced).  Returns (tokens int32
    [B, K+1] = accepted drafts, one drawn token, then -1; emit_count int32 [B])."""
    lib = load_library()
    if target_probs.dim() != 3 or draft_tokens.dim() != 2:
        raise ValueError("target_probs must be [B, K+1, V] and draft_tokens [B, K]")
    dev, dtype = target_probs.device, target_probs.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    B, K = draft_tokens.shape
    V = target_probs.shape[2]
    ps = _rows3(target_probs, "target_probs", B, K + 1, V, dtype, dev)
    qs = V if draft_probs is None else _rows3(draft_probs, "draft_probs", B, K, V, dtype, dev)
    _need(draft_tokens, "draft_tokens", torch.int32, dev)
    _need(uniforms, "uniforms", torch.float32, dev)
    _expect(uniforms, "uniforms", B * (K + 1))
    if draft_count is not None:
        _need(draft_count, "draft_count", torch.int32, dev)
        _expect(draft_count, "draft_count", B)
    if tokens is None:
        tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    else:
        _need(tokens, "tokens", torch.int32, dev)
        _expect(tokens, "tokens", B * (K + 1))
    if emit_count is None:
        emit_count = torch.empty(B, dtype=torch.int32, device=dev)
    else:
        _need(emit_count, "emit_count", torch.int32, dev)
        _expect(emit_count, "emit_count", B)
    _, ref = _descriptor(gdn_verify_shape, (B, K, V, _DTYPES[dtype], ps, qs))
    stream = _on_gpu(dev)
    if workspace is None:
        workspace = _scratch(lib.gdn_verify_workspace_bytes(ref), dev)
    else:
        _need(workspace, "workspace", None, dev)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.gdn_verify_drafts(ref, target_probs.data_ptr(), _addr(draft_probs), draft_tokens.data_ptr(),
                               uniforms.data_ptr(), _addr(draft_count), tokens.data_ptr(), emit_count.data_ptr(),
                               _addr(workspace), nbytes, stream)
    if st:
        _check(st)
    return tokens, emit_count


_ACTS = {"none": 0, "silu": 1, "sigmoid": 2}


def gdn_block_norm(y, *, gate=None, gate_act="silu", residual=None, residual_scale=1.0, post_weight=None,
                   next_weight=None, eps=1e-6, out=None, normed=None):
    """h = residual + residual_scale * act(gate) * RMSNorm_group(y) * post_weight and,
    with next_weight, normed = RMSNorm(h) * next_weight; every part but y is
    optional.  y, gate, residual [..., D] of one dtype; the group of the first
    norm is post_weight's length (D, or one of 16, 32, 64, 128 dividing D);
    next_weight [D].  ``out`` (h) may be y or residual.  Returns (h, normed or
    None)."""
    lib = load_library()
    dev, dtype = y.device, y.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    if gate_act not in _ACTS:
        raise ValueError(f"gate_act {gate_act!r} is not one of {sorted(_ACTS)}")
    if y.dim() < 1 or y.shape[-1] < 1:
        raise ValueError(f"y must be [..., D], got shape {tuple(y.shape)}")
    if gate is not None and gate_act == "none":
        raise ValueError("gate is given with gate_act 'none'")
    _need(y, "y")
    shape, D = y.shape, y.shape[-1]
    for t, n in ((gate, "gate"), (residual, "residual"), (out, "out"), (normed, "normed")):
        if t is not None:
            _need(t, n, dtype, dev)
            if t.shape != shape:
                raise ValueError(f"{n} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    group = D
    if post_weight is not None:
        _need(post_weight, "post_weight", dtype, dev)
        group = post_weight.numel()
        if group < 1 or D % group != 0:
            raise ValueError(f"post_weight has {group} elements, expected a divisor of {D}")
    if next_weight is not None:
        _need(next_weight, "next_weight", dtype, dev)
        _expect(next_weight, "next_weight", D)
        if normed is None:
            normed = torch.empty_like(y)
    elif normed is not None:
        raise ValueError("normed is given without next_weight")
    if out is None:
        out = torch.empty_like(y)
    _, ref = _descriptor(gdn_norm_shape, (y.numel() // D, D, group, _DTYPES[dtype],
                                          0 if gate is None else _ACTS[gate_act], float(residual_scale), float(eps)))
    stream = _on_gpu(dev)
    st = lib.gdn_block_norm(ref, y.data_ptr(), _addr(gate), _addr(residual), _addr(post_weight),
                            _addr(next_weight), out.data_ptr(), _addr(normed), stream)
    if st:
        _check(st)
    return out, normed


# ---------------------------------------------------------------------------
# Paged cache, beams
# ---------------------------------------------------------------------------
# The calls below are made once a layer and token: each first asks everything at once, and looks for what is wrong, to name
# it, only if something is.
def _tokens(t, name, dtype, index, ragged, H, d):
    """(elements between tokens, tokens, heads) of a [T, H, d] (ragged; also [1, T, H, d]) or [B, L, H, d] tensor whose
    tokens are evenly spaced and whole; any number of heads if H is None."""
    shape = t.shape
    n = len(shape)
    h, e = shape[-2:] if n > 2 else (-1, -1)
    if t.dtype is not dtype or t.get_device() != index or e != d or (h != H and H is not None) or \
            n != (3 if ragged else 4):
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, expected {'cpu' if index < 0 else f'cuda:{index}'}")
        if n == 4 and ragged and shape[0] == 1:
            return _tokens(t[0], name, dtype, index, ragged, H, d)
        if n != (3 if ragged else 4):
            raise ValueError(f"{name} must be {'[T, H, d] with cu_seqlens' if ragged else '[B, L, H, d]'}, "
                             f"got shape {tuple(shape)}")
        raise ValueError(f"{name} has shape {tuple(shape)}, expected heads {'of' if H is None else f'{H} of'} {d}")
    count = shape[0] if ragged else shape[0] * shape[1]
    if t.is_contiguous():
        return h * e, count, h
    s = t.stride()
    if (e > 1 and s[-1] != 1) or (h > 1 and s[-2] != e):
        raise ValueError(f"{name}'s heads must be contiguous within a token")
    if ragged:
        row = s[0] if count > 1 else h * e
    else:
        B, L = shape[:2]
        row = s[1] if L > 1 else (s[0] if B > 1 else h * e)
        if B > 1 and L > 1 and s[0] != L * row:
            raise ValueError(f"{name} must have evenly spaced tokens, got strides {tuple(s)}")
    if row < h * e:
        raise ValueError(f"{name}'s tokens overlap: strides {tuple(s)}")
    return row, count, h


_I32 = torch.int32


def _cache_common(k_cache, v_cache, block_table, cache_lens, cu_seqlens):
    """Checks shared by the cache's entry points; (device index, dtype, its code, k_cache's shape, N, max_pages)."""
    shape, dtype, index = k_cache.shape, k_cache.dtype, k_cache.get_device()
    code, table = _DTYPES.get(dtype), block_table.shape
    if code is None or len(shape) != 4 or len(table) != 2 or v_cache.shape != shape or v_cache.dtype is not dtype or \
            v_cache.get_device() != index or not (k_cache.is_contiguous() and v_cache.is_contiguous()) or \
            block_table.dtype is not _I32 or block_table.get_device() != index or not block_table.is_contiguous() or \
            cache_lens.dtype is not _I32 or cache_lens.get_device() != index or not cache_lens.is_contiguous() or \
            cache_lens.shape != table[:1] or shape[1] < 1 or shape[2] < 1:
        if len(shape) != 4 or len(table) != 2:
            raise ValueError("k_cache must be [num_pages, Hkv, page_size, d] and block_table [N, max_pages]")
        if code is None:
            raise TypeError(f"unsupported dtype {dtype}")
        dev = k_cache.device
        _need(k_cache, "k_cache", None, dev)
        _need(v_cache, "v_cache", dtype, dev)
        if v_cache.shape != shape:
            raise ValueError(f"v_cache has shape {tuple(v_cache.shape)}, k_cache {tuple(shape)}")
        _need(block_table, "block_table", _I32, dev)
        _need(cache_lens, "cache_lens", _I32, dev)
        if cache_lens.shape != table[:1]:
            raise ValueError(f"cache_lens has shape {tuple(cache_lens.shape)}, expected {(table[0],)}")
        raise ValueError(f"k_cache has shape {tuple(shape)}")
    N, max_pages = table
    if cu_seqlens is not None and (cu_seqlens.dtype is not _I32 or cu_seqlens.get_device() != index or
                                   cu_seqlens.shape != (N + 1,) or not cu_seqlens.is_contiguous()):
        _need(cu_seqlens, "cu_seqlens", _I32, k_cache.device)
        raise ValueError(f"cu_seqlens has shape {tuple(cu_seqlens.shape)}, expected {(N + 1,)}")
    return index, dtype, code, shape, N, max_pages


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(dev, call, *args):
    """call(*args, dev's stream): kernels start on the current device, so that is made dev where it is another."""
    stream = _on_gpu(dev)
    if _current_device() == dev.index:
        st = call(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = call(*args, stream)
    if st:
        _check(st)


def _like(t):
    """A new contiguous tensor of t's shape and type (a slice of wider rows may be the model)."""
    out = torch.empty_like(t)
    return out if out.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def gdn_cache_append(k, v, k_cache, v_cache, block_table, cache_lens, *, cu_seqlens=None, q=None, inv_freq=None,
                     positions=None, pair_axis=None, interleaved=False, q_out=None):
    """New keys and values into their pages, keys (and queries) rotated by their positions on the way.

    Dense k, v [N, L, Hkv, d], q [N, L, Hq, d]; ragged: [T, H, d] plus cu_seqlens int32 [N+1].  Tokens may be slices
    of wider rows.  k_cache, v_cache [num_pages, Hkv, page_size, d]; block_table int32 [N, max_pages]; cache_lens
    int32 [N] counts the new tokens.  inv_freq fp32 [rotary / 2] (None: nothing is rotated); positions int32
    [tokens] or [axes, tokens] (None: places in the cache); pair_axis int32 [rotary / 2] (which axis turns which
    pair).  ``interleaved`` pairs elements 2j, 2j + 1 instead of j, j + rotary / 2.  ``q_out`` may be q.
    Returns q_out (None without q)."""
    lib = load_library()
    ragged = cu_seqlens is not None
    index, dtype, code, shape, N, max_pages = _cache_common(k_cache, v_cache, block_table, cache_lens, cu_seqlens)
    pages, Hkv, page_size, d = shape
    ks, tokens, _ = _tokens(k, "k", dtype, index, ragged, Hkv, d)
    vs, nv, _ = _tokens(v, "v", dtype, index, ragged, Hkv, d)
    if nv != tokens or (not ragged and (k.shape[0] != N or v.shape != k.shape)):
        raise ValueError(f"k has shape {tuple(k.shape)}, v {tuple(v.shape)}, for {N} sequences")
    Hq, qs = Hkv, Hkv * d
    if q is not None:
        if inv_freq is None:
            raise ValueError("q is given without inv_freq: there is nothing to do with it")
        qs, nq, Hq = _tokens(q, "q", dtype, index, ragged, None, d)
        if nq != tokens or (not ragged and q.shape[:2] != k.shape[:2]):
            raise ValueError(f"q has shape {tuple(q.shape)}, k {tuple(k.shape)}")
        if Hq % Hkv != 0:
            raise ValueError(f"Hq={Hq} must be a multiple of Hkv={Hkv}")
        if q_out is None:
            q_out = _like(q)
        else:
            _need(q_out, "q_out", dtype, q.device)
            if q_out.shape != q.shape:
                raise ValueError(f"q_out has shape {tuple(q_out.shape)}, expected {tuple(q.shape)}")
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    rotary, axes = 0, 1
    if inv_freq is not None:
        rotary = 2 * inv_freq.numel()
        if inv_freq.dtype is not torch.float32 or inv_freq.get_device() != index or not inv_freq.is_contiguous() or \
                inv_freq.dim() != 1 or not 1 < rotary <= d:
            _need(inv_freq, "inv_freq", torch.float32, k_cache.device)
            raise ValueError(f"inv_freq has shape {tuple(inv_freq.shape)}, expected [rotary / 2] with rotary <= {d}")
    if positions is not None:
        _need(positions, "positions", _I32, k_cache.device)
        if inv_freq is None:
            raise ValueError("positions are given without inv_freq")
        axes = 1 if positions.dim() == 1 else positions.shape[0]
        if positions.dim() > 2 or axes < 1 or positions.shape[-1] != tokens:
            raise ValueError(f"positions has shape {tuple(positions.shape)}, expected [{tokens}] or [axes, {tokens}]")
    if pair_axis is not None:
        _need(pair_axis, "pair_axis", _I32, k_cache.device)
        _expect(pair_axis, "pair_axis", rotary // 2)
    elif axes > 1:
        raise ValueError(f"pair_axis is required with {axes} axes")
    _, ref = _descriptor(gdn_cache_shape, (N, tokens if ragged else k.shape[1], Hq, Hkv, d, code, page_size, pages,
                                           max_pages))
    _, how = _descriptor(gdn_append_shape, (qs, ks, vs, rotary, 1 if interleaved else 0, axes))
    _launch(k_cache.device, lib.gdn_cache_append, ref, how, _addr(q), k.data_ptr(), v.data_ptr(), _addr(inv_freq),
            _addr(positions), _addr(pair_axis), block_table.data_ptr(), cache_lens.data_ptr(), _addr(cu_seqlens),
            _addr(q_out), k_cache.data_ptr(), v_cache.data_ptr())
    return q_out


def gdn_cache_attention_workspace_bytes(shape: gdn_cache_shape, ragged: bool) -> int:
    """Bytes gdn_cache_attention needs for this shape (0: none)."""
    n = load_library().gdn_cache_attention_workspace_bytes(ctypes.byref(shape), int(bool(ragged)))
    if n == ctypes.c_size_t(-1).value:
        _check(GDN_ERR_INVALID_ARG)
    return int(n)


def gdn_cache_attention(q, k_cache, v_cache, block_table, cache_lens, *, cu_seqlens=None, scale=None, window=0, o=None,
                        workspace=None):
    """Causal attention of new tokens over the paged cache (their own keys included).

    Dense q [N, L, Hq, d]; ragged: [T, Hq, d] plus cu_seqlens int32 [N+1].  The cache as in gdn_cache_append; new token
    i of the L of a sequence has the place cache_lens - L + i and sees the keys up to it, with ``window`` only the
    last ``window`` of them.  ``scale`` is d^-1/2 unless given.  Returns o (q's shape, contiguous)."""
    lib = load_library()
    ragged = cu_seqlens is not None
    index, dtype, code, shape, N, max_pages = _cache_common(k_cache, v_cache, block_table, cache_lens, cu_seqlens)
    pages, Hkv, page_size, d = shape
    qs, tokens, Hq = _tokens(q, "q", dtype, index, ragged, None, d)
    if Hq < 1 or Hq % Hkv != 0:
        raise ValueError(f"Hq={Hq} must be a multiple of Hkv={Hkv}")
    if not ragged and q.shape[0] != N:
        raise ValueError(f"q has shape {tuple(q.shape)}, for {N} sequences")
    if o is None:
        o = _like(q)
    else:
        _need(o, "o", dtype, q.device)
        if o.shape != q.shape:
            raise ValueError(f"o has shape {tuple(o.shape)}, expected {tuple(q.shape)}")
    _, ref = _descriptor(gdn_cache_shape, (N, tokens if ragged else q.shape[1], Hq, Hkv, d, code, page_size, pages,
                                           max_pages))
    if not 0 <= window < 1 << 31:
        raise ValueError(f"window={window} must be in [0, 2^31)")
    dev = k_cache.device
    if workspace is None:   # an invalid shape is named by the call itself
        workspace = _scratch(lib.gdn_cache_attention_workspace_bytes(ref, ragged), dev)
    else:
        _need(workspace, "workspace", None, dev)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _launch(dev, lib.gdn_cache_attention, ref, q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(),
            block_table.data_ptr(), cache_lens.data_ptr(), _addr(cu_seqlens),
            d ** -0.5 if scale is None else float(scale), window, o.data_ptr(), _addr(workspace), nbytes)
    return o


def gdn_cache_copy_pages(k_cache, v_cache, src_pages, dst_pages):
    """Copies page src_pages[g, j] to page dst_pages[g, j] in both caches (int32, of one shape, [W] or [G, W] with W
    up to 64), as when a beam takes over the last, partly filled page of its parent.  Within a row of entries all
    reads come before all writes; a page that one row writes must not be read or written by another.  Negative
    numbers copy nothing."""
    lib = load_library()
    dev = k_cache.device
    _need(k_cache, "k_cache", None, dev)
    _need(v_cache, "v_cache", k_cache.dtype, dev)
    _need(src_pages, "src_pages", torch.int32, dev)
    _need(dst_pages, "dst_pages", torch.int32, dev)
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [num_pages, Hkv, page_size, d] of one shape")
    if src_pages.dim() not in (1, 2) or dst_pages.shape != src_pages.shape:
        raise ValueError(f"src_pages has shape {tuple(src_pages.shape)}, dst_pages {tuple(dst_pages.shape)}")
    G, W = (1, *src_pages.shape) if src_pages.dim() == 1 else src_pages.shape
    rows, apart = k_cache.shape[0], v_cache.data_ptr() - k_cache.data_ptr()
    if rows == 0 or src_pages.numel() == 0:
        return
    row = k_cache.numel() // rows * k_cache.element_size()
    _, ref = _descriptor(gdn_reorder_shape, (2, apart, apart, rows, rows, row, 0, G, W))
    _launch(dev, lib.gdn_state_reorder, ref, k_cache.data_ptr(), k_cache.data_ptr(), src_pages.data_ptr(),
            dst_pages.data_ptr())


def gdn_beam_workspace_bytes(shape: gdn_beam_shape) -> int:
    """Bytes gdn_beam_select needs for this shape."""
    n = load_library().gdn_beam_workspace_bytes(ctypes.byref(shape))
    if n == ctypes.c_size_t(-1).value:
        _check(GDN_ERR_INVALID_ARG)
    return int(n)


def gdn_beam_select(logits, scores, *, beams=None, finished=None, eos_token=-1, pad_token=0, tokens=None, parents=None,
                    new_scores=None, new_finished=None, workspace=None):
    """The best ``beams`` (None: W) continuations of W beams in each of B searches, by score + log softmax(logits).

    logits [B, W, V] (rows may be padded, evenly spaced), scores fp32 [B, W], finished bool [B, W] or None: a finished
    beam goes on with pad_token at its score.  Returns (tokens int32, parents int32, scores fp32, finished bool), each
    [B, beams], best first, ties to the lowest parent, then the lowest token; places that are left hold -1, -1,
    -infinity, True."""
    lib = load_library()
    if logits.dim() != 3:
        raise ValueError("logits must be [B, W, V]")
    dev, dtype = logits.device, logits.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    B, W, V = logits.shape
    K = W if beams is None else int(beams)
    row = _rows3(logits, "logits", B, W, V, dtype, dev)
    _need(scores, "scores", torch.float32, dev)
    if scores.shape != (B, W):
        raise ValueError(f"scores has shape {tuple(scores.shape)}, expected {(B, W)}")
    if finished is not None:
        _need(finished, "finished", torch.bool, dev)
        if finished.shape != (B, W):
            raise ValueError(f"finished has shape {tuple(finished.shape)}, expected {(B, W)}")
    if K < 1:
        raise ValueError(f"beams={K} < 1")
    outs = [tokens, parents, new_scores, new_finished]
    for i, kind in enumerate((_I32, _I32, torch.float32, torch.bool)):
        t = outs[i]
        if t is None:
            outs[i] = torch.empty_like(scores, dtype=kind) if K == W else torch.empty((B, K), dtype=kind, device=dev)
        elif t.dtype is not kind or t.device != dev or t.shape != (B, K) or not t.is_contiguous():
            name = ("tokens", "parents", "new_scores", "new_finished")[i]
            _need(t, name, kind, dev)
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(B, K)}")
    if not (-0x80000000 <= eos_token < 0x80000000 and -0x80000000 <= pad_token < 0x80000000):
        raise ValueError(f"eos_token={eos_token} or pad_token={pad_token} does not fit 32 bits")
    _, ref = _descriptor(gdn_beam_shape, (B, W, K, V, _DTYPES[dtype], int(eos_token), int(pad_token), row))
    if workspace is None:
        workspace = _scratch(lib.gdn_beam_workspace_bytes(ref), dev)
    else:
        _need(workspace, "workspace", None, dev)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _launch(dev, lib.gdn_beam_select, ref, logits.data_ptr(), scores.data_ptr(), _addr(finished), outs[0].data_ptr(),
            outs[1].data_ptr(), outs[2].data_ptr(), outs[3].data_ptr(), _addr(workspace), nbytes)
    return tuple(outs)


def gdn_state_reorder(state, parents, *, axis=0, out=None):
    """Rows of a state moved after a beam selection: row b * K + j of ``out`` becomes row b * W + parents[b, j] of
    ``state``, bitwise.  parents int32 [B, K]; the state has B * W rows along ``axis`` (the axes before it are
    layers) and any dtype, its rows a multiple of 16 bytes.  ``out`` may be the state itself (K = W).  Parents outside
    of [0, W) leave their row of ``out`` as it is.  Returns out."""
    lib = load_library()
    dev = state.device
    _need(state, "state")
    _need(parents, "parents", torch.int32, dev)
    if parents.dim() != 2:
        raise ValueError(f"parents must be [B, K], got shape {tuple(parents.shape)}")
    if not 0 <= axis < state.dim():
        raise ValueError(f"axis={axis} of a state with {state.dim()} axes")
    shape, (B, K) = state.shape, parents.shape
    rows = shape[axis]
    if rows % B != 0 if B else rows != 0:
        raise ValueError(f"state has {rows} rows for {B} searches")
    want = (*shape[:axis], B * K, *shape[axis + 1:])
    if out is None:
        out = torch.empty(want, dtype=state.dtype, device=dev)
    else:
        _need(out, "out", state.dtype, dev)
        if out.shape != want:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {want}")
    if parents.numel() == 0 or state.numel() == 0:
        return out
    layers = math.prod(shape[:axis])
    row = state.numel() // (layers * rows) * state.element_size()
    if row % 16 != 0:
        raise ValueError(f"a row of {row} bytes is not a multiple of 16")
    _, ref = _descriptor(gdn_reorder_shape, (layers, rows * row, B * K * row, rows, B * K, row, rows // B, B, K))
    _launch(dev, lib.gdn_state_reorder, ref, state.data_ptr(), out.data_ptr(), parents.data_ptr(), None)
    return out


def gdn_profile_enable(on: bool = True) -> None:
    """Turn per-kernel HIP-event timing inside the library on or off."""
    _check(load_library().gdn_profile_enable(int(bool(on))))


def gdn_profile_collect() -> dict:
    """{kernel name: (launches, total ms)} for the kernels timed since the last collect."""
    lib = load_library()
    n = 32
    names = (ctypes.c_char_p * n)()
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int32 * n)()
    k = lib.gdn_profile_collect(names, ms, cnt, n)
    return {names[i].decode(): (int(cnt[i]), float(ms[i])) for i in range(min(k, n))}


__all__ = ["gdn_profile_enable", "gdn_profile_collect", "load_library", "GdnError", "gdn_shape",
           "gdn_prefill_workspace_bytes", "gdn_prefill_chunked", "gdn_prefill_chunked_states",
           "gdn_prefill_chunked_noalloc", "GDN_NOALLOC_SCRATCH_BYTES",
           "gdn_prefill_chunked_ex", "gdn_recurrent_step_ex", "Prologue", "gdn_prologue",
           "gdn_recurrent_step", "gdn_replay_state_updates", "gdn_state_snapshot", "gdn_linear_workspace_bytes",
           "gdn_linear_prefill", "gdn_linear_step", "gdn_verify_drafts", "gdn_verify_shape", "gdn_block_norm",
           "gdn_norm_shape", "gdn_cache_append", "gdn_cache_attention_workspace_bytes", "gdn_cache_attention",
           "gdn_cache_copy_pages", "gdn_beam_workspace_bytes", "gdn_beam_select", "gdn_state_reorder",
           "gdn_cache_shape", "gdn_append_shape", "gdn_beam_shape", "gdn_reorder_shape", "EXPORTED", "LIB_PATH"]
