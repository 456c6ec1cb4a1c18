"""Thin Python binding of the C ABI in include/gdn_cpr.h.

Argument marshalling only.  Torch tensors become device pointers, the current
torch CUDA stream becomes the stream handle, and output buffers are allocated
with torch.  Every step of the CPR path runs in the library's CUDA kernels.
There is no fallback: if libgdn_cpr.so is missing, or no GPU is present, the
calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Dict, Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn_cpr.so")

GDN_F32, GDN_BF16 = 0, 1
GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_WORKSPACE = 0, 1, 2, 3, 4
GDN_ERR_TIMEOUT, GDN_ERR_DEVICE_INPUT = 5, 6
_STATUS = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED", 3: "GDN_ERR_CUDA",
           4: "GDN_ERR_WORKSPACE", 5: "GDN_ERR_TIMEOUT", 6: "GDN_ERR_DEVICE_INPUT"}

#: exported symbols of include/gdn_cpr.h
SYMBOLS = ("gdn_contract_id", "gdn_status_string", "gdn_num_chunk_states", "gdn_cpr_workspace_size",
           "gdn_cpr_forward", "gdn_decode_step", "gdn_cpr_forward_timed", "gdn_decode_step_timed",
           "gdn_decode_step_ex",
           "gdn_cpr_forward_noalloc", "gdn_contract_text", "gdn_contract_identity", "gdn_sha256_hex",
           "gdn_cpr_backward_workspace_size", "gdn_cpr_backward", "gdn_cpr_backward_timed",
           "gdn_read_device_status", "gdn_test_fault_injection",
           "gdn_conv_forward", "gdn_conv_backward_workspace_size", "gdn_conv_backward", "gdn_conv_step",
           "gdn_ssm_num_chunk_states", "gdn_ssm_forward",
           "gdn_ssm_backward_workspace_size", "gdn_ssm_backward", "gdn_ssm_step",
           "gdn_layer_norm_forward", "gdn_layer_norm_backward_workspace_size", "gdn_layer_norm_backward",
           "gdn_qk_norm_forward", "gdn_qk_norm_backward_workspace_size", "gdn_qk_norm_backward",
           "gdn_qk_norm_backward_ex",
           "gdn_glu_saved_size", "gdn_glu_forward_workspace_size", "gdn_glu_forward",
           "gdn_glu_backward_workspace_size", "gdn_glu_backward",
           "gdn_policy_loss_forward", "gdn_policy_loss_backward")

#: gdn_identity_kind_t
ID_SEMANTIC, ID_NUMERICAL_POLICY, ID_DEPLOYMENT = 0, 1, 2

#: tokens between two saved states of the selective scan (GDN_SSM_CHUNK)
SSM_CHUNK = 32

#: size of the fixed device array behind gdn_cpr_forward_noalloc (GDN_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 64 << 20


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_STATUS.get(status, status)} ({status})")
        self.status = status


class CacheStruct(ctypes.Structure):
    _fields_ = [("S_b", ctypes.c_void_p), ("R", ctypes.c_void_p), ("rscale", ctypes.c_void_p),
                ("kbuf", ctypes.c_void_p), ("vbuf", ctypes.c_void_p), ("abuf", ctypes.c_void_p),
                ("bbuf", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class SsmStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "dt", "B", "C", "z", "A", "D", "dt_bias", "cu_seqlens")] + \
               [(n, ctypes.c_int64) for n in ("x_stride", "dt_stride", "B_stride", "C_stride", "z_stride",
                                              "total_tokens")] + \
               [(n, ctypes.c_int32) for n in ("num_seqs", "channels", "groups", "states", "delta_softplus",
                                              "in_dtype")]


class QkNormStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")] + \
               [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "tokens")] + \
               [(n, ctypes.c_int32) for n in ("q_heads", "k_heads", "head_dim", "rot_dim", "interleaved", "unit")] + \
               [("eps", ctypes.c_float)] + [(n, ctypes.c_int32) for n in ("in_dtype", "w_dtype")]


class GluStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "w_gate", "w_up")] + \
               [(n, ctypes.c_int64) for n in ("x_stride", "gate_stride", "up_stride", "rows")] + \
               [(n, ctypes.c_int32) for n in ("width", "inner", "act", "in_dtype")]


class PolicyStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("logits", "targets", "old_logprob", "ref_logprob", "advantages")] + \
               [(n, ctypes.c_int64) for n in ("logits_stride", "rows")] + [("vocab", ctypes.c_int32)] + \
               [(n, ctypes.c_float) for n in ("clip_low", "clip_high", "kl_coef", "temperature")] + \
               [("in_dtype", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgdn_cpr.so (built by ``python -m gated_deltanet_cpr_delta_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with python -m gated_deltanet_cpr_delta_b200.build")
    lib = ctypes.CDLL(path)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.gdn_contract_id.restype = ctypes.c_char_p
    lib.gdn_contract_id.argtypes = []
    lib.gdn_contract_text.restype = i64
    lib.gdn_contract_text.argtypes = [ctypes.c_int, i32, i32, i32, ctypes.c_int, ctypes.c_int, ctypes.c_char_p, sz]
    lib.gdn_contract_identity.restype = ctypes.c_int
    lib.gdn_contract_identity.argtypes = [ctypes.c_int, i32, i32, i32, ctypes.c_int, ctypes.c_int, ctypes.c_char_p]
    lib.gdn_sha256_hex.restype = ctypes.c_int
    lib.gdn_sha256_hex.argtypes = [ctypes.c_void_p, sz, ctypes.c_char_p]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [ctypes.c_int]
    lib.gdn_num_chunk_states.restype = i64
    lib.gdn_num_chunk_states.argtypes = [P, i32, i32]
    lib.gdn_cpr_workspace_size.restype = sz
    lib.gdn_cpr_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32]
    lib.gdn_cpr_forward.restype = ctypes.c_int
    lib.gdn_cpr_forward.argtypes = [P, P, P, P, P, P, P, P, i32, i64, i32, i32, i32, i32, ctypes.c_int,
                                    ctypes.c_int, P, P, ctypes.POINTER(CacheStruct), P, sz, P]
    lib.gdn_decode_step.restype = ctypes.c_int
    lib.gdn_decode_step.argtypes = [P, P, P, P, P, ctypes.POINTER(CacheStruct), i32, i32, i32, i32, i32,
                                    ctypes.c_int, ctypes.c_int, P, P]
    lib.gdn_cpr_forward_timed.restype = ctypes.c_int
    lib.gdn_cpr_forward_timed.argtypes = lib.gdn_cpr_forward.argtypes + [P]
    lib.gdn_decode_step_timed.restype = ctypes.c_int
    lib.gdn_decode_step_timed.argtypes = lib.gdn_decode_step.argtypes + [P]
    lib.gdn_decode_step_ex.restype = ctypes.c_int
    lib.gdn_decode_step_ex.argtypes = lib.gdn_decode_step.argtypes[:-1] + [i32, P, P]
    lib.gdn_cpr_forward_noalloc.restype = ctypes.c_int
    lib.gdn_cpr_forward_noalloc.argtypes = [P, P, P, P, P, P, P, P, i32, i64, i32, i32, i32, i32, ctypes.c_int,
                                            ctypes.c_int, P, P, ctypes.POINTER(CacheStruct), P]
    lib.gdn_cpr_backward_workspace_size.restype = sz
    lib.gdn_cpr_backward_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32]
    lib.gdn_cpr_backward.restype = ctypes.c_int
    lib.gdn_cpr_backward.argtypes = [P, P, P, P, P, P, P, P, P, P, i32, i64, i32, i32, i32, i32, ctypes.c_int,
                                     P, P, P, P, P, P, P, sz, P]
    lib.gdn_cpr_backward_timed.restype = ctypes.c_int
    lib.gdn_cpr_backward_timed.argtypes = lib.gdn_cpr_backward.argtypes + [P]
    lib.gdn_read_device_status.restype = ctypes.c_int
    lib.gdn_read_device_status.argtypes = [P, P, P]
    lib.gdn_test_fault_injection.restype = ctypes.c_int
    lib.gdn_test_fault_injection.argtypes = [i32, i64]
    e = ctypes.c_int
    lib.gdn_conv_forward.restype = e
    lib.gdn_conv_forward.argtypes = [P, i64, P, P, P, P, i32, i64, i32, i32, i32, e, e, P, P, P, P]
    lib.gdn_conv_backward_workspace_size.restype = sz
    lib.gdn_conv_backward_workspace_size.argtypes = [i64, i32, i32, i32]
    lib.gdn_conv_backward.restype = e
    lib.gdn_conv_backward.argtypes = [P, i64, P, P, P, P, i64, P, P, i32, i64, i32, i32, i32, e, e, P, P, P, P, P, sz,
                                      P, P]
    lib.gdn_conv_step.restype = e
    lib.gdn_conv_step.argtypes = [P, i64, P, P, P, P, i32, i32, i32, i32, e, e, P, P]
    ssm = ctypes.POINTER(SsmStruct)
    lib.gdn_ssm_num_chunk_states.restype = i64
    lib.gdn_ssm_num_chunk_states.argtypes = [i64, i32]
    lib.gdn_ssm_forward.restype = e
    lib.gdn_ssm_forward.argtypes = [ssm, P, P, P, P, P, P]
    lib.gdn_ssm_backward_workspace_size.restype = sz
    lib.gdn_ssm_backward_workspace_size.argtypes = [i64, i32, i32, i32, i32]
    lib.gdn_ssm_backward.restype = e
    lib.gdn_ssm_backward.argtypes = [ssm, P, i64, P, P, P, P, P, P, P, P, P, P, P, P, sz, P, P]
    lib.gdn_ssm_step.restype = e
    lib.gdn_ssm_step.argtypes = [ssm, P, P, P, P]
    lib.gdn_layer_norm_forward.restype = e
    lib.gdn_layer_norm_forward.argtypes = [P, i64, P, P, ctypes.c_float, i64, i32, e, e, P, P, P, P]
    lib.gdn_layer_norm_backward_workspace_size.restype = sz
    lib.gdn_layer_norm_backward_workspace_size.argtypes = [i64, i32]
    lib.gdn_layer_norm_backward.restype = e
    lib.gdn_layer_norm_backward.argtypes = [P, i64, P, i64, P, P, P, i64, i32, e, e, P, P, P, P, sz, P]
    qk, pol = ctypes.POINTER(QkNormStruct), ctypes.POINTER(PolicyStruct)
    lib.gdn_qk_norm_forward.restype = e
    lib.gdn_qk_norm_forward.argtypes = [qk, P, P, P]
    lib.gdn_qk_norm_backward_workspace_size.restype = sz
    lib.gdn_qk_norm_backward_workspace_size.argtypes = [i64, i32]
    lib.gdn_qk_norm_backward.restype = e
    lib.gdn_qk_norm_backward.argtypes = [qk, P, i64, P, i64, P, P, P, P, P, sz, P]
    lib.gdn_qk_norm_backward_ex.restype = e
    lib.gdn_qk_norm_backward_ex.argtypes = [qk, e, P, i64, P, i64, P, P, P, P, P, sz, P]
    glu = ctypes.POINTER(GluStruct)
    lib.gdn_glu_saved_size.restype = i64
    lib.gdn_glu_saved_size.argtypes = [i64, i32]
    lib.gdn_glu_forward_workspace_size.restype = sz
    lib.gdn_glu_forward_workspace_size.argtypes = [glu]
    lib.gdn_glu_forward.restype = e
    lib.gdn_glu_forward.argtypes = [glu, P, P, P, sz, P, P]
    lib.gdn_glu_backward_workspace_size.restype = sz
    lib.gdn_glu_backward_workspace_size.argtypes = [glu]
    lib.gdn_glu_backward.restype = e
    lib.gdn_glu_backward.argtypes = [glu, P, i64, P, P, P, P, e, P, sz, P, P]
    lib.gdn_policy_loss_forward.restype = e
    lib.gdn_policy_loss_forward.argtypes = [pol, P, P, P, P]
    lib.gdn_policy_loss_backward.restype = e
    lib.gdn_policy_loss_backward.argtypes = [pol, P, P, P, P, P, P]
    _lib = lib
    return lib


def _dt(t: torch.dtype) -> int:
    if t == torch.float32:
        return GDN_F32
    if t == torch.bfloat16:
        return GDN_BF16
    raise ValueError(f"unsupported dtype {t}")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _event_array(events, n: int):
    """torch.cuda.Event list -> C array of cudaEvent_t handles (events must
    have been recorded once so that the CUDA event exists)."""
    if len(events) != n:
        raise ValueError(f"need {n} events")
    handles = [e.cuda_event for e in events]
    if any(h == 0 for h in handles):
        raise ValueError("record each event once before passing it (creates the CUDA event)")
    return (ctypes.c_void_p * n)(*handles)


def _check(st: int, what: str):
    if st != 0:
        raise GdnError(st, what)


def gdn_contract_id() -> str:
    return load_library().gdn_contract_id().decode()


def gdn_contract_text(kind: int, d_k: int, d_v: int, C: int, in_dtype: int, out_dtype: int) -> str:
    lib = load_library()
    n = lib.gdn_contract_text(kind, d_k, d_v, C, in_dtype, out_dtype, None, 0)
    if n < 0:
        raise GdnError(1, "gdn_contract_text")
    buf = ctypes.create_string_buffer(n + 1)
    lib.gdn_contract_text(kind, d_k, d_v, C, in_dtype, out_dtype, buf, n + 1)
    return buf.value.decode()


def gdn_contract_identity(kind: int, d_k: int, d_v: int, C: int, in_dtype: int, out_dtype: int) -> str:
    out = ctypes.create_string_buffer(65)
    _check(load_library().gdn_contract_identity(kind, d_k, d_v, C, in_dtype, out_dtype, out), "gdn_contract_identity")
    return out.value.decode()


def gdn_sha256_hex(data: bytes) -> str:
    out = ctypes.create_string_buffer(65)
    buf = ctypes.create_string_buffer(bytes(data), len(data))
    _check(load_library().gdn_sha256_hex(buf, len(data), out), "gdn_sha256_hex")
    return out.value.decode()


def gdn_num_chunk_states(cu_seqlens_host: Sequence[int], C: int) -> int:
    arr = (ctypes.c_int32 * len(cu_seqlens_host))(*[int(x) for x in cu_seqlens_host])
    n = load_library().gdn_num_chunk_states(arr, len(cu_seqlens_host) - 1, C)
    if n < 0:
        raise GdnError(1, "gdn_num_chunk_states")
    return int(n)


def gdn_cpr_workspace_size(total_tokens: int, num_seqs: int, H: int, d_k: int, d_v: int, C: int) -> int:
    return int(load_library().gdn_cpr_workspace_size(total_tokens, num_seqs, H, d_k, d_v, C))


def new_cache(N: int, H: int, d_k: int, d_v: int, C: int, dtype: torch.dtype, device="cuda",
              state: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Allocate a decode cache (gdn_cache_t layout).  With ``state`` [N,H,d_v,d_k]
    it starts at a chunk boundary with that state, otherwise at zero.  The
    running state is ``rscale * R``.  ``status`` is the decode step's device
    status word (one int32, starts at GDN_OK).  ``pos_host`` is a host copy of
    each sequence's buffer position (CPU int32 [N]): :func:`gdn_decode_step`
    skips the resync launch on steps where no buffer can fill."""
    S = torch.zeros(N, H, d_v, d_k, dtype=torch.float32, device=device) if state is None else state.clone()
    return dict(S_b=S, R=S.clone(), rscale=torch.ones(N, H, dtype=torch.float32, device=device),
                kbuf=torch.zeros(N, H, C, d_k, dtype=dtype, device=device),
                vbuf=torch.zeros(N, H, C, d_v, dtype=dtype, device=device),
                abuf=torch.zeros(N, H, C, dtype=torch.float32, device=device),
                bbuf=torch.zeros(N, H, C, dtype=torch.float32, device=device),
                pos=torch.zeros(N, H, dtype=torch.int32, device=device),
                status=torch.zeros(1, dtype=torch.int32, device=device),
                pos_host=torch.zeros(N, dtype=torch.int32))


def _set_pos_host(cache: Dict[str, torch.Tensor], cu_seqlens_host, C: int):
    """After a prefill into ``cache``: each sequence's position is L mod C."""
    cu = [int(x) for x in cu_seqlens_host]
    cache["pos_host"] = torch.tensor([(cu[n + 1] - cu[n]) % C for n in range(len(cu) - 1)], dtype=torch.int32)


def _cache_struct(c: Dict[str, torch.Tensor]) -> CacheStruct:
    st = c.get("status")
    return CacheStruct(*[c[n].data_ptr() for n in ("S_b", "R", "rscale", "kbuf", "vbuf", "abuf", "bbuf", "pos")],
                       st.data_ptr() if st is not None else None)


def read_device_status(workspace: Optional[torch.Tensor] = None, device=None) -> int:
    """The device status word of the last forward / backward that used
    ``workspace`` (None: the no-allocation forward's fixed array), read after
    the current stream has run that call (this synchronises the stream)."""
    dev = workspace.device if workspace is not None else torch.device("cuda", torch.cuda.current_device())
    out = torch.empty(1, dtype=torch.int32, device=dev)
    _check(load_library().gdn_read_device_status(_ptr(workspace), _ptr(out), _stream(dev)),
           "gdn_read_device_status")
    return int(out.item())


def set_fault_injection(mode: int, wait_clocks: int = 1 << 31) -> None:
    """Failure-detection hook (process-wide; mode 0 = off): see
    gdn_test_fault_injection in include/gdn_cpr.h."""
    _check(load_library().gdn_test_fault_injection(mode, wait_clocks), "gdn_test_fault_injection")


def gdn_cpr_forward(q, k, v, alpha, beta, cu_seqlens, C: int, *, cu_seqlens_host=None, state_in=None,
                    out_dtype=None, cache_out: Optional[Dict[str, torch.Tensor]] = None, workspace=None,
                    o=None, chunk_states=None, events=None):
    """CPR forward (prefill / trainer forward).

    q, k [T,H,d_k], v [T,H,d_v] (bf16 or fp32); alpha, beta [T,H] fp32;
    cu_seqlens int32 device [N+1] (``cu_seqlens_host``: the same values on the
    host; read back with a sync when omitted); state_in [N,H,d_v,d_k] fp32 or None.
    Returns (o [T,H,d_v] in out_dtype (default: q.dtype), chunk_states).
    ``events``: optional 6 torch.cuda.Events, recorded around the kernels
    (calls gdn_cpr_forward_timed).
    """
    lib = load_library()
    T, H, dk = k.shape
    dv = v.shape[2]
    if cu_seqlens_host is None:
        cu_seqlens_host = cu_seqlens.cpu().tolist()
    cu_h = (ctypes.c_int32 * len(cu_seqlens_host))(*[int(x) for x in cu_seqlens_host])
    N = len(cu_seqlens_host) - 1
    out_dtype = q.dtype if out_dtype is None else out_dtype
    dev = k.device
    if o is None:
        o = torch.empty(T, H, dv, dtype=out_dtype, device=dev)
    if chunk_states is None:
        ns = lib.gdn_num_chunk_states(cu_h, N, C)
        if ns < 0:
            raise GdnError(1, "gdn_num_chunk_states")
        chunk_states = torch.empty(ns, H, dv, dk, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(lib.gdn_cpr_workspace_size(T, N, H, dk, dv, C), dtype=torch.uint8, device=dev)
    cs = _cache_struct(cache_out) if cache_out is not None else None
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state_in),
            _ptr(cu_seqlens), cu_h, N, T, H, dk, dv, C, _dt(q.dtype), _dt(out_dtype),
            _ptr(o), _ptr(chunk_states), ctypes.byref(cs) if cs is not None else None,
            _ptr(workspace), workspace.numel(), _stream(dev))
    if events is None:
        st = lib.gdn_cpr_forward(*args)
    else:
        st = lib.gdn_cpr_forward_timed(*args, _event_array(events, 6))
    _check(st, "gdn_cpr_forward")
    if cache_out is not None:
        _set_pos_host(cache_out, cu_seqlens_host, C)
    return o, chunk_states


def gdn_cpr_backward_workspace_size(total_tokens: int, num_seqs: int, H: int, d_k: int, d_v: int, C: int) -> int:
    return int(load_library().gdn_cpr_backward_workspace_size(total_tokens, num_seqs, H, d_k, d_v, C))


def gdn_cpr_backward(q, k, v, alpha, beta, dO, chunk_states, cu_seqlens, C: int, *, cu_seqlens_host=None,
                     dstate_out=None, workspace=None, grads=None, events=None):
    """CPR backward: gradients of sum(dO * o) for the forward of the same inputs.

    q, k, v, alpha, beta, cu_seqlens: as given to :func:`gdn_cpr_forward`;
    dO [T,H,d_v] in q's dtype; chunk_states: that forward's chunk states;
    dstate_out [N,H,d_v,d_k] fp32 or None: the loss gradient for each
    sequence's final state (a later part's dstate_in, when a sequence is split).
    Returns (dq, dk, dv, dalpha, dbeta, dstate_in), all fp32.  ``grads``: an
    optional tuple of those six tensors to write into.  ``events``: optional
    4 torch.cuda.Events recorded around the kernels (gdn_cpr_backward_timed)."""
    lib = load_library()
    T, H, dk = k.shape
    dv = v.shape[2]
    if cu_seqlens_host is None:
        cu_seqlens_host = cu_seqlens.cpu().tolist()
    cu_h = (ctypes.c_int32 * len(cu_seqlens_host))(*[int(x) for x in cu_seqlens_host])
    N = len(cu_seqlens_host) - 1
    dev = k.device
    if grads is None:
        f32 = dict(dtype=torch.float32, device=dev)
        grads = (torch.empty(T, H, dk, **f32), torch.empty(T, H, dk, **f32), torch.empty(T, H, dv, **f32),
                 torch.empty(T, H, **f32), torch.empty(T, H, **f32), torch.empty(N, H, dv, dk, **f32))
    if workspace is None:
        workspace = torch.empty(lib.gdn_cpr_backward_workspace_size(T, N, H, dk, dv, C), dtype=torch.uint8,
                                device=dev)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(dO), _ptr(chunk_states), _ptr(dstate_out),
            _ptr(cu_seqlens), cu_h, N, T, H, dk, dv, C, _dt(q.dtype),
            *[_ptr(g) for g in grads], _ptr(workspace), workspace.numel(), _stream(dev))
    if events is None:
        st = lib.gdn_cpr_backward(*args)
    else:
        st = lib.gdn_cpr_backward_timed(*args, _event_array(events, 4))
    _check(st, "gdn_cpr_backward")
    return grads


def gdn_decode_step(q, k, v, alpha, beta, cache: Dict[str, torch.Tensor], C: int, *, out_dtype=None, o=None,
                    events=None):
    """One decode token per sequence.  q,k [N,H,d_k], v [N,H,d_v]; alpha, beta [N,H].
    ``cache`` (from :func:`new_cache` or a forward's ``cache_out``) is updated in place.
    ``events``: optional 3 torch.cuda.Events around the two kernels.  With the
    cache's ``pos_host`` (kept by :func:`new_cache`, the forwards and this call)
    the resync launch is skipped on steps where no sequence's buffer fills
    (gdn_decode_step_ex's hint); without it the resync is always launched."""
    lib = load_library()
    N, H, dk = k.shape
    dv = v.shape[2]
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if o is None:
        o = torch.empty(N, H, dv, dtype=out_dtype, device=k.device)
    cs = _cache_struct(cache)
    ph = cache.get("pos_host")
    ph = ph.numpy() if ph is not None else None  # numpy view of the CPU tensor: cheap host arithmetic
    may_resync = 1 if ph is None else int((ph >= C - 1).any())
    st = lib.gdn_decode_step_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), ctypes.byref(cs), N, H, dk,
                                dv, C, _dt(q.dtype), _dt(out_dtype), _ptr(o), may_resync, _stream(k.device),
                                _event_array(events, 3) if events is not None else None)
    _check(st, "gdn_decode_step")
    if ph is not None:
        ph += 1
        ph[ph >= C] = 0
    return o


def gdn_cpr_forward_noalloc(q, k, v, alpha, beta, cu_seqlens, C: int, *, cu_seqlens_host=None, state_in=None,
                            out_dtype=None, cache_out: Optional[Dict[str, torch.Tensor]] = None, o=None,
                            chunk_states=None):
    """CPR forward whose workspace is the library's fixed device array (see
    gdn_cpr_forward_noalloc in include/gdn_cpr.h): for callers that cannot
    allocate device memory when they call.  Same arguments and results as
    :func:`gdn_cpr_forward` without ``workspace``; ``o`` and ``chunk_states``
    should be passed in by such callers (they are allocated here only when
    omitted).  Calls that overlap on the GPU race on the shared array."""
    lib = load_library()
    T, H, dk = k.shape
    dv = v.shape[2]
    if cu_seqlens_host is None:
        cu_seqlens_host = cu_seqlens.cpu().tolist()
    cu_h = (ctypes.c_int32 * len(cu_seqlens_host))(*[int(x) for x in cu_seqlens_host])
    N = len(cu_seqlens_host) - 1
    out_dtype = q.dtype if out_dtype is None else out_dtype
    dev = k.device
    if o is None:
        o = torch.empty(T, H, dv, dtype=out_dtype, device=dev)
    if chunk_states is None:
        chunk_states = torch.empty(gdn_num_chunk_states(cu_seqlens_host, C), H, dv, dk, dtype=torch.float32,
                                   device=dev)
    cs = _cache_struct(cache_out) if cache_out is not None else None
    st = lib.gdn_cpr_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state_in),
                                     _ptr(cu_seqlens), cu_h, N, T, H, dk, dv, C, _dt(q.dtype), _dt(out_dtype),
                                     _ptr(o), _ptr(chunk_states), ctypes.byref(cs) if cs is not None else None,
                                     _stream(dev))
    _check(st, "gdn_cpr_forward_noalloc")
    if cache_out is not None:
        _set_pos_host(cache_out, cu_seqlens_host, C)
    return o, chunk_states


# ------------------------------------------------------------------ layer operators
# The short causal convolution, the selective state space scan and layer norm
# (include/gdn_cpr.h, "layer operators").  Token tensors may be row-strided
# views (slices of one projection's output); everything else is contiguous.
# All tensors of a call lie on one GPU, which need not be the current one.
# The checks are written to cost little: a single-token step runs a few microseconds.

_F32 = torch.float32
_DT = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


def _dense(what: str, name: str, t: torch.Tensor, dtype: torch.dtype, shape, dev: int) -> int:
    """The address of a contiguous tensor of this type and shape on device `dev`."""
    if t.dtype is not dtype:
        raise ValueError(f"{what}: {name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: {name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{what}: tensors on cuda:{dev} and {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous")
    return t.data_ptr()


def _opt(what: str, name: str, t: Optional[torch.Tensor], dtype: torch.dtype, shape, dev: int):
    return None if t is None else _dense(what, name, t, dtype, shape, dev)


def _out(what: str, name: str, t: Optional[torch.Tensor], dtype: torch.dtype, shape, dev: int, like=None):
    """(tensor, address) of an output: the caller's, or a new one (``like``: a tensor of its shape, and perhaps type)."""
    if t is None:
        # empty_like takes half the time of empty with a type and a device; views of a wider tensor come out dense, but for
        # unusual orders of their axes
        if like is not None and like.dtype is dtype:
            t = torch.empty_like(like)
            if t.is_contiguous():
                return t, t.data_ptr()
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _dense(what, name, t, dtype, shape, dev)


def _rows(what: str, name: str, t: torch.Tensor, dtype: torch.dtype, shape, dev: int):
    """(address, elements between rows) of a token tensor whose rows are dense."""
    if t.dtype is not dtype:
        raise ValueError(f"{what}: {name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: {name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{what}: tensors on cuda:{dev} and {t.device}")
    width = 1
    for n in shape[1:]:
        width *= n
    if t.is_contiguous():
        return t.data_ptr(), width
    w = 1
    for n, st in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and st != w:
            raise ValueError(f"{what}: the rows of {name} must be contiguous")
        w *= n
    if shape[0] > 1 and t.stride(0) < width:
        raise ValueError(f"{what}: the rows of {name} overlap")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else width


def _type(what: str, t: torch.Tensor) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise ValueError(f"{what}: unsupported dtype {t.dtype}")
    return dt


def _gpu(what: str, t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what}: tensors must be on a CUDA device")
    return dev


def _call(dev: int, what: str, fn, *args) -> None:
    """Run fn(*args, stream) on the current stream of device `dev`, with that device current."""
    if torch.cuda.current_device() == dev:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != 0:
        raise GdnError(st, what)


def _sequences(what: str, cu: Optional[torch.Tensor], dev: int):
    """(address, number of sequences) of device offsets; None: one sequence."""
    if cu is None:
        return None, 1
    if cu.dtype is not torch.int32 or cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError(f"{what}: cu_seqlens must be a contiguous int32 vector")
    return _dense(what, "cu_seqlens", cu, torch.int32, cu.shape, dev), cu.shape[0] - 1


@functools.lru_cache(maxsize=1024)
def _scratch_size(name: str, *sizes: int) -> int:
    return int(getattr(load_library(), name)(*sizes))


def _scratch(what: str, workspace: Optional[torch.Tensor], nbytes: int, dev: int):
    """(tensor to keep alive, address, bytes)"""
    if workspace is None:
        w = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        return w, w.data_ptr(), nbytes
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"{what}: workspace must be contiguous and on cuda:{dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _conv_sizes(what, x, weight):
    xs, ws = x.shape, weight.shape
    if len(xs) != 2 or len(ws) != 2 or ws[0] != xs[1]:
        raise ValueError(f"{what}: x must be [tokens, channels] and weight [channels, width]")
    return xs[0], xs[1], ws[1]


def gdn_conv_forward(x, weight, cu_seqlens=None, *, bias=None, state_in=None, silu: bool = True, y=None,
                     state_out=None, status=None):
    """Short causal convolution of a packed batch (gdn_conv_forward).

    x [T, channels] (bf16 or fp32, rows may be strided); weight [channels, W], bias [channels] or
    None (bf16 or fp32), W in 2..4; cu_seqlens int32 device [N+1] or None (one
    sequence); state_in [N, W-1, channels] in x's dtype or None for zeros.
    Returns (y [T, channels], state_out [N, W-1, channels]): the last inputs, for
    :func:`gdn_conv_step` or the next part of the sequence.  ``y`` and
    ``state_out``: optional buffers to write; rows of y outside every sequence
    keep their contents.  ``status``: an optional int32 that records bad offsets."""
    what = "gdn_conv_forward"
    T, D, W = _conv_sizes(what, x, weight)
    dt, wt = x.dtype, weight.dtype
    ti, wi = _type(what, x), _type(what, weight)
    pc, N = _sequences(what, cu_seqlens, x.get_device())
    dev = _gpu(what, x)
    px, ldx = _rows(what, "x", x, dt, (T, D), dev)
    pw = _dense(what, "weight", weight, wt, (D, W), dev)
    y, py = _out(what, "y", y, dt, (T, D), dev, x)
    state_out, ps = _out(what, "state_out", state_out, dt, (N, W - 1, D), dev)
    _call(dev, what, load_library().gdn_conv_forward, px, ldx, pw, _opt(what, "bias", bias, wt, (D,), dev),
          _opt(what, "state_in", state_in, dt, (N, W - 1, D), dev), pc, N, T, D, W, silu, ti, wi, py, ps,
          _opt(what, "status", status, torch.int32, (1,), dev))
    return y, state_out


def gdn_conv_backward(x, weight, dy, cu_seqlens=None, *, bias=None, state_in=None, silu: bool = True,
                      dstate_out=None, workspace=None, grads=None, status=None):
    """Gradients of sum(dy y) + sum(dstate_out state_out) for :func:`gdn_conv_forward` of the same inputs.

    dy [T, channels] in x's dtype (rows may be strided); dstate_out [N, W-1, channels] fp32 or None.
    Returns (dx in x's dtype, dweight, dbias (None without a bias), dstate_in), the
    last three fp32.  ``grads``: an optional tuple of those four to write into."""
    what = "gdn_conv_backward"
    T, D, W = _conv_sizes(what, x, weight)
    dt, wt = x.dtype, weight.dtype
    ti, wi = _type(what, x), _type(what, weight)
    dev = _gpu(what, x)
    pc, N = _sequences(what, cu_seqlens, dev)
    if grads is None:
        grads = (torch.empty((T, D), dtype=dt, device=dev), torch.empty((D, W), dtype=_F32, device=dev),
                 None if bias is None else torch.empty((D,), dtype=_F32, device=dev),
                 torch.empty((N, W - 1, D), dtype=_F32, device=dev))
    dx, dw, db, ds = grads
    px, ldx = _rows(what, "x", x, dt, (T, D), dev)
    pg, ldg = _rows(what, "dy", dy, dt, (T, D), dev)
    keep, ws, nbytes = _scratch(what, workspace, _scratch_size("gdn_conv_backward_workspace_size", T, N, D, W), dev)
    _call(dev, what, load_library().gdn_conv_backward, px, ldx, _dense(what, "weight", weight, wt, (D, W), dev),
          _opt(what, "bias", bias, wt, (D,), dev), _opt(what, "state_in", state_in, dt, (N, W - 1, D), dev), pg, ldg,
          _opt(what, "dstate_out", dstate_out, _F32, (N, W - 1, D), dev), pc, N, T, D, W, silu, ti, wi,
          _dense(what, "dx", dx, dt, (T, D), dev), _dense(what, "dweight", dw, _F32, (D, W), dev),
          _opt(what, "dbias", db, _F32, (D,), dev), _dense(what, "dstate_in", ds, _F32, (N, W - 1, D), dev), ws, nbytes,
          _opt(what, "status", status, torch.int32, (1,), dev))
    return grads


def gdn_conv_step(x, weight, state, *, bias=None, silu: bool = True, y=None, state_out=None):
    """One token per sequence: x [N, channels], state [N, W-1, channels] (from
    :func:`gdn_conv_forward`), updated in place or written to ``state_out``.  Returns y [N, channels]."""
    what = "gdn_conv_step"
    N, D, W = _conv_sizes(what, x, weight)
    dt, wt = x.dtype, weight.dtype
    ti, wi = _type(what, x), _type(what, weight)
    dev = _gpu(what, x)
    px, ldx = _rows(what, "x", x, dt, (N, D), dev)
    y, py = _out(what, "y", y, dt, (N, D), dev, x)
    ps = _dense(what, "state", state, dt, (N, W - 1, D), dev)
    _call(dev, what, load_library().gdn_conv_step, px, ldx, _dense(what, "weight", weight, wt, (D, W), dev),
          _opt(what, "bias", bias, wt, (D,), dev), ps,
          ps if state_out is None else _dense(what, "state_out", state_out, dt, (N, W - 1, D), dev), N, D, W, silu, ti,
          wi, py)
    return y


def _ssm_struct(what, x, dt, A, B, C, pc, N, D, z, dt_bias, dt_softplus) -> SsmStruct:
    if x.dim() != 2 or B.dim() != 3:
        raise ValueError(f"{what}: x must be [tokens, channels] and B [tokens, groups, states]")
    T, ch = x.shape
    _, G, S = B.shape
    ty = x.dtype
    ti = _type(what, x)
    dev = x.get_device()
    tc, ts, cs = (T, ch), (T, G, S), (ch,)
    px, lx = _rows(what, "x", x, ty, tc, dev)
    pd, ld = _rows(what, "dt", dt, ty, tc, dev)
    pB, lB = _rows(what, "B", B, ty, ts, dev)
    pC, lC = _rows(what, "C", C, ty, ts, dev)
    pz, lz = (None, 0) if z is None else _rows(what, "z", z, ty, tc, dev)
    s = SsmStruct(px, pd, pB, pC, pz, _dense(what, "A", A, _F32, (ch, S), dev), _opt(what, "D", D, _F32, cs, dev),
                  _opt(what, "dt_bias", dt_bias, _F32, cs, dev), pc, lx, ld, lB, lC, lz, T, N, ch, G, S, dt_softplus, ti)
    _gpu(what, x)
    return s


def gdn_ssm_num_chunk_states(total_tokens: int, num_seqs: int) -> int:
    n = load_library().gdn_ssm_num_chunk_states(total_tokens, num_seqs)
    if n < 0:
        raise GdnError(1, "gdn_ssm_num_chunk_states")
    return int(n)


def gdn_ssm_forward(x, dt, A, B, C, cu_seqlens=None, *, D=None, z=None, dt_bias=None, dt_softplus: bool = True,
                    state_in=None, save_states: bool = False, y=None, state_out=None, chunk_states=None,
                    status=None):
    """Selective state space scan of a packed batch (gdn_ssm_forward): per channel c of group g
        delta = softplus(dt + dt_bias),  h = exp(delta A) h + delta x B[g],  y = (h . C[g] + D x) silu(z)

    x, dt, z [T, channels], B, C [T, groups, states] (bf16 or fp32, rows may be strided); A [channels, states], D,
    dt_bias [channels] fp32; z, D, dt_bias may be None; states in {16, 32, 64}; cu_seqlens int32
    device [N+1] or None (one sequence); state_in [N, channels, states] fp32 or None.
    Returns (y, state_out, chunk_states).  chunk_states (with ``save_states``; else
    None) is what :func:`gdn_ssm_backward` reads."""
    what = "gdn_ssm_forward"
    dev = x.get_device()
    pc, N = _sequences(what, cu_seqlens, dev)
    s = _ssm_struct(what, x, dt, A, B, C, pc, N, D, z, dt_bias, dt_softplus)
    T, ch, S, ty = s.total_tokens, s.channels, s.states, x.dtype
    y, py = _out(what, "y", y, ty, (T, ch), dev, x)
    state_out, ps = _out(what, "state_out", state_out, _F32, (N, ch, S), dev)
    saved = (T // SSM_CHUNK + N, ch, S)
    if chunk_states is None and save_states:
        chunk_states = torch.empty(saved, dtype=_F32, device=dev)
    _call(dev, what, load_library().gdn_ssm_forward, s, _opt(what, "state_in", state_in, _F32, (N, ch, S), dev),
          py, ps, _opt(what, "chunk_states", chunk_states, _F32, saved, dev), _opt(what, "status", status, torch.int32, (1,), dev))
    return y, state_out, chunk_states


def gdn_ssm_backward(x, dt, A, B, C, dy, chunk_states, cu_seqlens=None, *, D=None, z=None, dt_bias=None,
                     dt_softplus: bool = True, dstate_out=None, workspace=None, grads=None, status=None):
    """Gradients of sum(dy y) + sum(dstate_out state_out) for :func:`gdn_ssm_forward` of the same inputs.

    dy [T, channels] in x's dtype (rows may be strided); chunk_states: that forward's; dstate_out
    [N, channels, states] fp32 or None.  Returns (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dstate_in): dx, ddt, dB, dC and
    dz in x's dtype, the others fp32; dD, dz and ddt_bias are None where the
    forward had no D, z or dt_bias.  ``grads``: an optional tuple of those nine to write into."""
    what = "gdn_ssm_backward"
    dev = x.get_device()
    pc, N = _sequences(what, cu_seqlens, dev)
    s = _ssm_struct(what, x, dt, A, B, C, pc, N, D, z, dt_bias, dt_softplus)
    T, ch, G, S, ty = s.total_tokens, s.channels, s.groups, s.states, x.dtype
    tc, ts, st, cs = (T, ch), (T, G, S), (N, ch, S), (ch,)
    if grads is None:
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        grads = (new(tc, ty), new(tc, ty), new((ch, S), _F32), new(ts, ty), new(ts, ty),
                 None if D is None else new(cs, _F32), None if z is None else new(tc, ty),
                 None if dt_bias is None else new(cs, _F32), new(st, _F32))
    dx, ddt, dA, dB, dC, dD, dz, dbias, ds = grads
    if z is not None and dz is None:
        raise ValueError(f"{what}: dz is needed with z")
    pg, ldg = _rows(what, "dy", dy, ty, tc, dev)
    keep, ws, nbytes = _scratch(what, workspace, _scratch_size("gdn_ssm_backward_workspace_size", T, N, ch, G, S), dev)
    _call(dev, what, load_library().gdn_ssm_backward, s, pg, ldg,
          _dense(what, "chunk_states", chunk_states, _F32, (T // SSM_CHUNK + N, ch, S), dev),
          _opt(what, "dstate_out", dstate_out, _F32, st, dev), _dense(what, "dx", dx, ty, tc, dev),
          _dense(what, "ddt", ddt, ty, tc, dev), _dense(what, "dA", dA, _F32, (ch, S), dev),
          _dense(what, "dB", dB, ty, ts, dev), _dense(what, "dC", dC, ty, ts, dev), _opt(what, "dD", dD, _F32, cs, dev),
          _opt(what, "dz", dz, ty, tc, dev), _opt(what, "ddt_bias", dbias, _F32, cs, dev),
          _dense(what, "dstate_in", ds, _F32, st, dev), ws, nbytes, _opt(what, "status", status, torch.int32, (1,), dev))
    return grads


def gdn_ssm_step(x, dt, A, B, C, state, *, D=None, z=None, dt_bias=None, dt_softplus: bool = True, y=None,
                 state_out=None):
    """One token per sequence: x, dt, z [N, channels], B, C [N, groups, states]; state [N, channels, states] fp32 (from
    :func:`gdn_ssm_forward`), updated in place or written to ``state_out``.  Returns y [N, channels]."""
    what = "gdn_ssm_step"
    s = _ssm_struct(what, x, dt, A, B, C, None, x.shape[0], D, z, dt_bias, dt_softplus)
    dev = x.get_device()
    shape = (s.num_seqs, s.channels, s.states)
    y, py = _out(what, "y", y, x.dtype, shape[:2], dev, x)
    ps = _dense(what, "state", state, _F32, shape, dev)
    _call(dev, what, load_library().gdn_ssm_step, s, ps,
          ps if state_out is None else _dense(what, "state_out", state_out, _F32, shape, dev),
          py)
    return y


def _rows2d(what: str, name: str, t: torch.Tensor) -> torch.Tensor:
    """[.., width] as [rows, width] without a copy."""
    if t.dim() == 2:
        return t
    if t.dim() < 1:
        raise ValueError(f"{what}: {name} must have at least one axis")
    if t.numel() == 0:
        return t.reshape(t.numel() // max(1, t.shape[-1]), t.shape[-1])
    try:
        return t.view(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{what}: the leading axes of {name} must be one stride apart") from None


def gdn_layer_norm_forward(x, weight, *, bias=None, eps: float = 1e-5, y=None):
    """Layer norm over the last axis (gdn_layer_norm_forward): x [.., width] (bf16 or fp32, rows
    may be strided), weight [width] and bias [width] or None (bf16 or fp32).  A recurrence's output
    [T, H, d_v] is normalised per head.  Returns (y in x's shape and dtype, mean, rstd fp32 [..])."""
    what = "gdn_layer_norm_forward"
    x2 = _rows2d(what, "x", x)
    R, D = x2.shape
    dt, wt, shape = x.dtype, weight.dtype, x.shape
    ti, wi = _type(what, x), _type(what, weight)
    dev = _gpu(what, x)
    px, ldx = _rows(what, "x", x2, dt, (R, D), dev)
    y, py = _out(what, "y", y, dt, shape, dev, x)
    mean, rstd = torch.empty((2,) + tuple(shape[:-1]), dtype=_F32, device=dev).unbind(0)
    _call(dev, what, load_library().gdn_layer_norm_forward, px, ldx, _dense(what, "weight", weight, wt, (D,), dev),
          _opt(what, "bias", bias, wt, (D,), dev), eps, R, D, ti, wi, py, mean.data_ptr(), rstd.data_ptr())
    return y, mean, rstd


def gdn_layer_norm_backward(x, weight, dy, mean, rstd, *, workspace=None, grads=None):
    """Gradients of sum(dy y) for :func:`gdn_layer_norm_forward`: dy in x's shape and dtype,
    mean and rstd as that call returned them.  Returns (dx in x's dtype, dweight,
    dbias), the last two fp32, summed over the rows.  ``grads``: an optional tuple of those three to
    write into (dbias may be None)."""
    what = "gdn_layer_norm_backward"
    x2, g2 = _rows2d(what, "x", x), _rows2d(what, "dy", dy)
    R, D = x2.shape
    dt, wt, shape = x.dtype, weight.dtype, x.shape
    ti, wi = _type(what, x), _type(what, weight)
    dev = _gpu(what, x)
    if dy.shape != shape:
        raise ValueError(f"{what}: dy must have shape {tuple(shape)}, not {tuple(dy.shape)}")
    if grads is None:
        grads = (torch.empty(shape, dtype=dt, device=dev), torch.empty((D,), dtype=_F32, device=dev),
                 torch.empty((D,), dtype=_F32, device=dev))
    dx, dw, db = grads
    px, ldx = _rows(what, "x", x2, dt, (R, D), dev)
    pg, ldg = _rows(what, "dy", g2, dt, (R, D), dev)
    keep, ws, nbytes = _scratch(what, workspace, _scratch_size("gdn_layer_norm_backward_workspace_size", R, D), dev)
    _call(dev, what, load_library().gdn_layer_norm_backward, px, ldx, pg, ldg,
          _dense(what, "weight", weight, wt, (D,), dev), _dense(what, "mean", mean, _F32, shape[:-1], dev),
          _dense(what, "rstd", rstd, _F32, shape[:-1], dev), R, D, ti, wi, _dense(what, "dx", dx, dt, shape, dev),
          _dense(what, "dweight", dw, _F32, (D,), dev), _opt(what, "dbias", db, _F32, (D,), dev), ws, nbytes)
    return grads


def _heads(what: str, name: str, t: torch.Tensor, dtype: torch.dtype, shape, dev: int):
    """As _rows, for [tokens, heads, head_dim]; the usual views of a projection without a walk over the strides."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        a, b, c = t.stride()
        if c == 1 and b == shape[2] and a >= b * shape[1] and shape[0] > 1:
            return t.data_ptr(), a
    return _rows(what, name, t, dtype, shape, dev)


def _qk_struct(what, q, k, q_weight, k_weight, positions, inv_freq, interleaved, l2, eps, dev):
    if q.dim() != 3 or k.dim() != 3 or q.shape[0] != k.shape[0] or q.shape[2] != k.shape[2]:
        raise ValueError(f"{what}: q must be [tokens, q_heads, head_dim] and k [tokens, k_heads, head_dim]")
    if (positions is None) != (inv_freq is None):
        raise ValueError(f"{what}: positions and inv_freq go together")
    T, Hq, d = q.shape
    Hk, ty = k.shape[1], q.dtype
    weight = q_weight if q_weight is not None else k_weight
    wt = ty if weight is None else weight.dtype
    ti = _type(what, q)
    pq, lq = _heads(what, "q", q, ty, (T, Hq, d), dev)
    pk, lk = _heads(what, "k", k, ty, (T, Hk, d), dev)
    rot, pp, pf = 0, None, None
    if positions is not None:
        if inv_freq.dim() != 1:
            raise ValueError(f"{what}: inv_freq must be a vector")
        rot = 2 * inv_freq.shape[0]
        pp = _dense(what, "positions", positions, torch.int32, (T,), dev)
        pf = _dense(what, "inv_freq", inv_freq, _F32, inv_freq.shape, dev)
    return QkNormStruct(pq, pk, _opt(what, "q_weight", q_weight, wt, (d,), dev), _opt(what, "k_weight", k_weight, wt, (d,), dev),
                        pp, pf, lq, lk, T, Hq, Hk, d, rot, interleaved, l2, eps, ti, _DT.get(wt, -1))


def gdn_qk_norm_forward(q, k, *, q_weight=None, k_weight=None, positions=None, inv_freq=None, interleaved: bool = False,
                        l2: bool = False, eps: float = 1e-6, q_out=None, k_out=None):
    """Norm of every query's and key's head with the position rotation in the same pass (gdn_qk_norm_forward).

    q [T, q_heads, d], k [T, k_heads, d] (bf16 or fp32; tokens may be strided, so slices of one projection's output
    do), d even and at most 256; q_weight, k_weight [d] or None (bf16 or fp32, one type); positions int32 [T] and inv_freq
    fp32 [rot / 2] turn the first rot dimensions in pairs (i, i + rot / 2), or (2 i, 2 i + 1) with
    ``interleaved``; both None: no rotation.  ``l2``: rows of unit length (as the recurrence takes
    them) instead of unit mean square.  A decode step's tokens are rows like any other.  Returns
    (q_out, k_out), dense, in the inputs' shapes and type."""
    what = "gdn_qk_norm_forward"
    dev = _gpu(what, q)
    s = _qk_struct(what, q, k, q_weight, k_weight, positions, inv_freq, interleaved, l2, eps, dev)
    q_out, pq = _out(what, "q_out", q_out, q.dtype, q.shape, dev, q)
    k_out, pk = _out(what, "k_out", k_out, q.dtype, k.shape, dev, k)
    _call(dev, what, load_library().gdn_qk_norm_forward, s, pq, pk)
    return q_out, k_out


def gdn_qk_norm_backward(q, k, dq_out, dk_out, *, q_weight=None, k_weight=None, positions=None, inv_freq=None,
                         interleaved: bool = False, l2: bool = False, eps: float = 1e-6, workspace=None, grads=None):
    """Gradients of sum(dq_out q_out) + sum(dk_out k_out) for :func:`gdn_qk_norm_forward` of the same inputs.

    dq_out, dk_out in q's and k's shapes, in their type or both fp32, as :func:`gdn_cpr_backward` returns them (tokens may
    be strided).  Returns (dq, dk, dq_weight, dk_weight): the first two in the inputs' type, the others fp32, summed over tokens and heads, None without the
    weight.  ``grads``: an optional tuple of those four to write into."""
    what = "gdn_qk_norm_backward"
    dev = _gpu(what, q)
    s = _qk_struct(what, q, k, q_weight, k_weight, positions, inv_freq, interleaved, l2, eps, dev)
    T, d, ty = s.tokens, s.head_dim, q.dtype
    gt = _F32 if dq_out.dtype is _F32 else ty
    pgq, lgq = _heads(what, "dq_out", dq_out, gt, q.shape, dev)
    pgk, lgk = _heads(what, "dk_out", dk_out, gt, k.shape, dev)
    if grads is None:
        dqw = dkw = None
        if q_weight is not None and k_weight is not None:
            dqw, dkw = torch.empty((2, d), dtype=_F32, device=dev).unbind(0)
        elif q_weight is not None:
            dqw = torch.empty((d,), dtype=_F32, device=dev)
        elif k_weight is not None:
            dkw = torch.empty((d,), dtype=_F32, device=dev)
        grads = (None, None, dqw, dkw)
    dq, dk, dqw, dkw = grads
    dq, pdq = _out(what, "dq", dq, ty, q.shape, dev, q)
    dk, pdk = _out(what, "dk", dk, ty, k.shape, dev, k)
    keep, ws, nbytes = None, None, 0
    if dqw is not None or dkw is not None:
        keep, ws, nbytes = _scratch(what, workspace, _scratch_size("gdn_qk_norm_backward_workspace_size", T, d), dev)
    _call(dev, what, load_library().gdn_qk_norm_backward_ex, s, _DT[gt], pgq, lgq, pgk, lgk, pdq, pdk, _opt(what, "dq_weight", dqw, _F32, (d,), dev),
          _opt(what, "dk_weight", dkw, _F32, (d,), dev), ws, nbytes)
    return dq, dk, dqw, dkw


#: gdn_glu_t.act
ACTS = {"silu": 0, "gelu": 1}


def _glu_struct(what, x, w_gate, w_up, act, dev):
    x2 = _rows2d(what, "x", x)
    if w_gate.dim() != 2 or w_gate.shape[1] != x2.shape[1]:
        raise ValueError(f"{what}: x must be [.., width] and w_gate, w_up [inner, width]")
    if act not in ACTS:
        raise ValueError(f"{what}: act must be one of {sorted(ACTS)}, not {act!r}")
    R, D = x2.shape
    F, ty = w_gate.shape[0], x.dtype
    ti = _type(what, x)
    px, lx = _rows(what, "x", x2, ty, (R, D), dev)
    pg, lg = _rows(what, "w_gate", w_gate, ty, (F, D), dev)
    pu, lu = _rows(what, "w_up", w_up, ty, (F, D), dev)
    return GluStruct(px, pg, pu, lx, lg, lu, R, D, F, ACTS[act], ti)


def _glu_scratch(what, workspace, size, s, dev):
    """As _scratch, for sizes that follow from the addresses; nothing is allocated where nothing is needed."""
    if torch.cuda.current_device() == dev:
        n = size(s)
    else:
        with torch.cuda.device(dev):
            n = size(s)
    return _scratch(what, workspace, n, dev) if n else (None, None, 0)


def gdn_glu_forward(x, w_gate, w_up, *, act: str = "silu", save: bool = False, h=None, saved=None, workspace=None, status=None):
    """The gated feed-forward block's projections, activation and product (gdn_glu_forward):
        h = act(x w_gate^T) (x w_up^T)

    x [.., width], w_gate, w_up [inner, width], bf16 (rows may be strided: the weights may be halves of one matrix); ``act``
    "silu" or "gelu" (tanh form).  Returns (h [.., inner], saved): saved (with ``save``; else None) is what
    :func:`gdn_glu_backward` reads, 6 bytes per element of h.  Single tokens of a decode step are rows like any
    other; the order of h's sums goes by the number of rows and by inner.  ``status``: an optional int32 that records a wait that ran out."""
    what = "gdn_glu_forward"
    dev = _gpu(what, x)
    s = _glu_struct(what, x, w_gate, w_up, act, dev)
    R, F = s.rows, s.inner
    shape = x.shape[:-1] + (F,)
    if h is None:
        h = x.new_empty(shape)
    ph = _dense(what, "h", h, x.dtype, shape, dev)
    if saved is None and save:
        saved = torch.empty((6 * R * F,), dtype=torch.uint8, device=dev)
    lib = load_library()
    keep, ws, nbytes = _glu_scratch(what, workspace, lib.gdn_glu_forward_workspace_size, s, dev)
    _call(dev, what, lib.gdn_glu_forward, s, ph, _opt(what, "saved", saved, torch.uint8, (6 * R * F,), dev), ws, nbytes,
          _opt(what, "status", status, torch.int32, (1,), dev))
    return h, saved


def gdn_glu_backward(x, w_gate, w_up, dh, saved, *, act: str = "silu", workspace=None, grads=None, status=None):
    """Gradients of sum(dh h) for :func:`gdn_glu_forward` of the same inputs with ``save``.

    dh [.., inner] in x's type (rows may be strided).  Returns (dx in x's shape, dw_gate, dw_up), in x's type.
    ``grads``: an optional tuple of those three to write into; what is None in it is allocated.  The weights' gradients
    may then be fp32, both: the one that is given decides.  They hold the sums; the operands' own rounding to bf16 stays."""
    what = "gdn_glu_backward"
    dev = _gpu(what, x)
    s = _glu_struct(what, x, w_gate, w_up, act, dev)
    R, D, F, ty = s.rows, s.width, s.inner, x.dtype
    if dh.shape != x.shape[:-1] + (F,):
        raise ValueError(f"{what}: dh must have shape {tuple(x.shape[:-1]) + (F,)}, not {tuple(dh.shape)}")
    pd, ld = _rows(what, "dh", _rows2d(what, "dh", dh), ty, (R, F), dev)
    dx, dwg, dwu = grads if grads is not None else (None, None, None)
    wt = dwg.dtype if dwg is not None else dwu.dtype if dwu is not None else ty
    dx, pdx = _out(what, "dx", dx, ty, x.shape, dev, x)
    dwg, pdg = _out(what, "dw_gate", dwg, wt, (F, D), dev, w_gate)
    dwu, pdu = _out(what, "dw_up", dwu, wt, (F, D), dev, w_up)
    lib = load_library()
    keep, ws, nbytes = _glu_scratch(what, workspace, lib.gdn_glu_backward_workspace_size, s, dev)
    _call(dev, what, lib.gdn_glu_backward, s, pd, ld, _dense(what, "saved", saved, torch.uint8, (6 * R * F,), dev),
          pdx, pdg, pdu, _type(what, dwg), ws, nbytes, _opt(what, "status", status, torch.int32, (1,), dev))
    return dx, dwg, dwu


def _policy_struct(what, logits, targets, old_logprob, advantages, ref_logprob, clip_low, clip_high, kl_coef, temperature, dev):
    if logits.dim() != 2:
        raise ValueError(f"{what}: logits must be [rows, vocab]")
    if (old_logprob is None) != (advantages is None) or (ref_logprob is not None and old_logprob is None):
        raise ValueError(f"{what}: old_logprob and advantages go together, and with ref_logprob")
    R, V = logits.shape
    ti = _type(what, logits)
    pz, lz = _rows(what, "logits", logits, logits.dtype, (R, V), dev)
    return PolicyStruct(pz, _dense(what, "targets", targets, torch.int64, (R,), dev),
                        _opt(what, "old_logprob", old_logprob, _F32, (R,), dev),
                        _opt(what, "ref_logprob", ref_logprob, _F32, (R,), dev),
                        _opt(what, "advantages", advantages, _F32, (R,), dev), lz, R, V, clip_low, clip_high, kl_coef,
                        temperature, ti)


def gdn_policy_loss_forward(logits, targets, *, old_logprob=None, advantages=None, ref_logprob=None, clip_low: float = 0.2,
                            clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0, loss=None, logprob=None,
                            status=None):
    """Clipped policy loss with a KL term for each row of logits [rows, vocab] (gdn_policy_loss_forward):
        logprob = log_softmax(logits / temperature)[target],  ratio = exp(logprob - old_logprob)
        loss = -min(ratio A, clip(ratio, 1 - clip_low, 1 + clip_high) A) + kl_coef (e^g - g - 1),  g = ref_logprob - logprob

    logits bf16 or fp32 (rows may be strided); targets int64 [rows], negative: the row takes no part (its results are 0);
    old_logprob, advantages, ref_logprob fp32 [rows]; temperature at least 2^-100.  ref_logprob None or kl_coef 0: no KL term; old_logprob and advantages None: the
    log-probabilities alone, as a rollout records them.  Returns (loss or None, logprob), fp32 [rows].  A row's
    log-probability has the same bits in every batch and in :func:`gdn_policy_loss_backward`.
    ``status``: an optional int32 that records a target outside the vocabulary."""
    what = "gdn_policy_loss_forward"
    dev = _gpu(what, logits)
    s = _policy_struct(what, logits, targets, old_logprob, advantages, ref_logprob, clip_low, clip_high, kl_coef, temperature, dev)
    shape = (s.rows,)
    if logprob is None and old_logprob is None:
        logprob = torch.empty_like(targets, dtype=_F32)
    logprob, pl = _out(what, "logprob", logprob, _F32, shape, dev, old_logprob)
    po = None
    if old_logprob is not None:
        loss, po = _out(what, "loss", loss, _F32, shape, dev, old_logprob)
    elif loss is not None:
        raise ValueError(f"{what}: a loss needs old_logprob and advantages")
    _call(dev, what, load_library().gdn_policy_loss_forward, s, po, pl, _opt(what, "status", status, torch.int32, (1,), dev))
    return loss, logprob


def gdn_policy_loss_backward(logits, targets, dloss, *, old_logprob, advantages, ref_logprob=None, clip_low: float = 0.2,
                             clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0, dlogits=None, loss=None,
                             logprob=None, status=None):
    """The logits' gradient of sum(dloss loss) for :func:`gdn_policy_loss_forward` of the same inputs, and that call's
    results: a training step whose weights ``dloss`` (fp32 [rows]) are known is this call alone.

    Returns (dlogits [rows, vocab] in the logits' type, loss, logprob).  ``dlogits`` may be the (dense) logits
    themselves: the gradient then takes their place."""
    what = "gdn_policy_loss_backward"
    dev = _gpu(what, logits)
    s = _policy_struct(what, logits, targets, old_logprob, advantages, ref_logprob, clip_low, clip_high, kl_coef, temperature, dev)
    shape = (s.rows,)
    dlogits, pd = _out(what, "dlogits", dlogits, logits.dtype, logits.shape, dev, logits)
    loss, po = _out(what, "loss", loss, _F32, shape, dev, old_logprob)
    logprob, pl = _out(what, "logprob", logprob, _F32, shape, dev, old_logprob)
    _call(dev, what, load_library().gdn_policy_loss_backward, s, _dense(what, "dloss", dloss, _F32, shape, dev), pd, po, pl,
          _opt(what, "status", status, torch.int32, (1,), dev))
    return dlogits, loss, logprob
