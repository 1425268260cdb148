"""Gated DeltaNet-2 token-mixer core for GB300 (sm_103a): thin Python binding of libgdn2.so.

Every step of the computation runs in the library's CUDA kernels; this module only marshals
arguments (device pointers, sizes, the current CUDA stream) from torch tensors to the C ABI declared
in include/gdn2.h, and raises on a non-zero status. torch provides device memory and streams only.

The binding fails loudly: importing it raises if libgdn2.so has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn2.so")

GDN2_OK, GDN2_ERR_INVALID_ARG, GDN2_ERR_UNSUPPORTED = 0, -1, -2
GDN2_ERR_MISALIGNED, GDN2_ERR_WORKSPACE, GDN2_ERR_CUDA, GDN2_ERR_TIMEOUT = -3, -4, -5, -6
GDN2_F32, GDN2_BF16 = 0, 1
PATHS = {"auto": 0, "simt": 1, "tcgen05": 2}

#: names of the extern "C" functions exported by libgdn2.so (all declared in include/gdn2.h)
EXPORTS = (
    "gdn2_status_string", "gdn2_version", "gdn2_chunk_fwd_workspace_size",
    "gdn2_chunk_fwd_workspace_size_path", "gdn2_chunk_fwd", "gdn2_chunk_fwd_path",
    "gdn2_recurrent_step", "gdn2_last_device_status", "gdn2_set_wait_limit", "gdn2_selftest_umma",
    "gdn2_chunk_fwd_noalloc", "gdn2_recurrent_update", "gdn2_fg2_inputs", "gdn2_mixer_prologue",
    "gdn2_mixer_epilogue", "gdn2_backward_workspace_size", "gdn2_backward",
    "gdn2_backward_recurrent_workspace_size", "gdn2_backward_recurrent", "gdn2_mixer_decode_step",
    "gdn2_ssm_prologue", "gdn2_ssm_prologue_backward_workspace_size", "gdn2_ssm_prologue_backward",
    "gdn2_ssm_chunk_fwd_workspace_size", "gdn2_ssm_chunk_fwd", "gdn2_ssm_backward_workspace_size", "gdn2_ssm_backward",
    "gdn2_ssm_decode_step", "gdn2_block_norm", "gdn2_block_norm_backward_workspace_size", "gdn2_block_norm_backward",
    "gdn2_attn_prologue", "gdn2_attn_prologue_paged", "gdn2_attn_prologue_backward_workspace_size", "gdn2_attn_prologue_backward",
    "gdn2_attn_decode_workspace_size", "gdn2_attn_decode", "gdn2_pages_append", "gdn2_pages_append_active", "gdn2_pages_fork",
    "gdn2_pages_fork_active", "gdn2_pages_release", "gdn2_pages_copy",
)


class Gdn2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()' "
            "or python gated_deltanet_mixer_gdn2_gb300/_build.py)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
    sig = {
        "gdn2_status_string": (ctypes.c_char_p, [I]),
        "gdn2_version": (I, []),
        "gdn2_chunk_fwd_workspace_size": (Z, [I] * 7 + [I]),
        "gdn2_chunk_fwd_workspace_size_path": (Z, [I] + [I] * 7 + [I]),
        "gdn2_chunk_fwd": (I, [P] * 9 + [I] * 7 + [F, I, P, Z, P]),
        "gdn2_chunk_fwd_path": (I, [I] + [P] * 9 + [I] * 7 + [F, I, P, Z, P]),
        "gdn2_recurrent_step": (I, [P] * 8 + [I] * 5 + [F, I, P]),
        "gdn2_last_device_status": (I, [P]),
        "gdn2_set_wait_limit": (None, [L]),
        "gdn2_selftest_umma": (I, [I, I, P, P, P, P]),
        "gdn2_chunk_fwd_noalloc": (I, [P] * 9 + [I] * 7 + [F, I, P]),
        "gdn2_recurrent_update": (I, [P] * 7 + [I, P, I, P] + [I] * 6 + [F, I, P]),
        "gdn2_fg2_inputs": (I, [P] * 7 + [I] * 5 + [I, P]),
        "gdn2_mixer_prologue": (I, [P] * 18 + [I] * 7 + [I, P]),
        "gdn2_mixer_epilogue": (I, [P, P, P, F, P] + [I] * 4 + [I, P]),
        "gdn2_backward_workspace_size": (Z, [I] * 6 + [I]),
        "gdn2_backward": (I, [P] * 16 + [I] * 6 + [F, I, P, Z, P]),
        "gdn2_backward_recurrent_workspace_size": (Z, [I] * 6 + [I]),
        "gdn2_backward_recurrent": (I, [P] * 16 + [I] * 6 + [F, I, P, Z, P]),
        "gdn2_mixer_decode_step": (I, [P] * 15 + [F, P] + [I] * 6 + [F, I, P]),
        "gdn2_ssm_prologue": (I, [P, L, P, L] + [P] * 9 + [I] * 5 + [I, P]),
        "gdn2_ssm_prologue_backward_workspace_size": (Z, [I] * 5 + [I]),
        "gdn2_ssm_prologue_backward": (I, [P, L, P, L] + [P] * 5 + [P, L, P, P, P, L, P, L] + [P] * 4 + [I] * 5 + [I, P, Z, P]),
        "gdn2_ssm_chunk_fwd_workspace_size": (Z, [I] * 8 + [I]),
        "gdn2_ssm_chunk_fwd": (I, [I, P, L, P, P, P, L, P, L] + [P] * 5 + [I] * 6 + [I, P, Z, P]),
        "gdn2_ssm_backward_workspace_size": (Z, [I] * 8 + [I]),
        "gdn2_ssm_backward": (I, [I, P, L, P, P, P, L, P, L, P, P, P, L, P, P, P, L, P, P, P, L, P, L, P, P] + [I] * 6 +
                              [I, P, Z, P]),
        "gdn2_ssm_decode_step": (I, [P, L, P, L] + [P] * 7 + [I, P, I, P] + [I] * 5 + [I, P]),
        "gdn2_block_norm": (I, [P] * 8 + [L, I, I, F, I, P]),
        "gdn2_block_norm_backward_workspace_size": (Z, [L, I]),
        "gdn2_block_norm_backward": (I, [P] * 14 + [L, I, I, F, I, P, Z, P]),
        "gdn2_attn_prologue": (I, [P, L, P, L] + [P] * 7 + [I] * 7 + [F, I, P]),
        "gdn2_attn_prologue_paged": (I, [P, L, P, L, P, L] + [P] * 11 + [I] * 4 + [I] * 7 + [F, I, P]),
        "gdn2_attn_prologue_backward_workspace_size": (Z, [I] * 4),
        "gdn2_attn_prologue_backward": (I, [P, L, P, L] + [P] * 5 + [P, L] * 4 + [P, P] + [I] * 7 + [F, I, P, Z, P]),
        "gdn2_attn_decode_workspace_size": (Z, [I] * 7 + [I]),
        "gdn2_attn_decode": (I, [P, L] + [P] * 5 + [I] * 4 + [P] + [I] * 5 + [F, I, I, P, Z, P]),
        "gdn2_pages_append": (I, [P] * 5 + [I, P] + [I] * 5 + [P]),
        "gdn2_pages_append_active": (I, [P] * 5 + [I, P, P] + [I] * 5 + [P]),
        "gdn2_pages_fork": (I, [P] * 8 + [I] * 5 + [P]),
        "gdn2_pages_fork_active": (I, [P] * 9 + [I] * 5 + [P]),
        "gdn2_pages_release": (I, [P] * 4 + [I] * 4 + [P]),
        "gdn2_pages_copy": (I, [P, P, I, P, P, I, I, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.gdn2_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != GDN2_OK:
        raise Gdn2Error(status, what)


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return GDN2_BF16
    if t.dtype == torch.float32:
        return GDN2_F32
    raise TypeError(f"unsupported token dtype {t.dtype} (float32 or bfloat16)")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def gdn2_version() -> int:
    return lib.gdn2_version()


def gdn2_chunk_fwd_workspace_size(B, T, Hk, Hv, dk, dv, C=64, dtype=GDN2_BF16, path="auto") -> int:
    return lib.gdn2_chunk_fwd_workspace_size_path(PATHS[path], B, T, Hk, Hv, dk, dv, C, dtype)


def gdn2_chunk_fwd(q, k, v, g, b, w, o, initial_state=None, final_state=None, *, C=64, scale=1.0,
                   workspace=None, path="auto", stream=None):
    """Chunked forward (C ABI gdn2_chunk_fwd_path). Writes `o` and, if given, `final_state`.

    q, k: [B, T, H_k, d_k]; v, w: [B, T, H_v, d_v]; g, b: [B, T, H_v, d_k]; o: like v;
    states: [B, H_v, d_k, d_v] float32. `workspace`: a uint8 CUDA tensor of at least
    gdn2_chunk_fwd_workspace_size(...) bytes (allocated here when None).
    """
    import torch

    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = _dtype_code(q)
    for t in (k, v, g, b, w, o):
        if t.dtype != q.dtype:
            raise TypeError("all token tensors and o must share one dtype")
    for t in (initial_state, final_state):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("states are float32")
    need = gdn2_chunk_fwd_workspace_size(B, T, Hk, Hv, dk, dv, C, dt, path)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = lib.gdn2_chunk_fwd_path(PATHS[path], _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w),
                                 _ptr(initial_state), _ptr(final_state), _ptr(o), B, T, Hk, Hv, dk, dv,
                                 C, float(scale), dt, _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "gdn2_chunk_fwd")
    return o, final_state


def gdn2_chunk_fwd_noalloc(q, k, v, g, b, w, o, initial_state=None, final_state=None, *, C=64, scale=1.0,
                           stream=None):
    """Chunked forward without a caller workspace (C ABI gdn2_chunk_fwd_noalloc): for callers that
    cannot allocate device memory; the library's fixed 32 MiB device array serves as workspace."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    st = lib.gdn2_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(initial_state),
                                    _ptr(final_state), _ptr(o), B, T, Hk, Hv, dk, dv, C, float(scale),
                                    _dtype_code(q), _stream(stream))
    _check(st, "gdn2_chunk_fwd_noalloc")
    return o, final_state


def gdn2_recurrent_step(q, k, v, g, b, w, state, o, *, scale=1.0, stream=None):
    """One decode token (C ABI gdn2_recurrent_step); updates `state` in place and writes `o`.

    q, k: [B, H_k, d_k]; v, w: [B, H_v, d_v]; g, b: [B, H_v, d_k]; state: [B, H_v, d_k, d_v] fp32.
    """
    B, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    dt = _dtype_code(q)
    st = lib.gdn2_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(state),
                                 _ptr(o), B, Hk, Hv, dk, dv, float(scale), dt, _stream(stream))
    _check(st, "gdn2_recurrent_step")
    return o


def gdn2_recurrent_update(q, k, v, g, b, w, state, o, slots=None, *, scale=1.0, stream=None):
    """N tokens per call (C ABI gdn2_recurrent_update); updates `state` in place and writes `o`.

    q, k: [B, N, H_k, d_k]; v, w, o: [B, N, H_v, d_v]; g, b: [B, N, H_v, d_k]. state: float32 or
    bfloat16, [B, H_v, d_k, d_v], or a pool [n_slots, H_v, d_k, d_v] when `slots` (int32 [B]) is given.
    """
    import torch

    B, N, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    sdt = _dtype_code(state)
    n_slots = state.shape[0] if slots is not None else 0
    if slots is not None and slots.dtype != torch.int32:
        raise TypeError("slots must be int32")
    st = lib.gdn2_recurrent_update(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(state), sdt,
                                   _ptr(slots), n_slots, _ptr(o), B, N, Hk, Hv, dk, dv, float(scale),
                                   _dtype_code(q), _stream(stream))
    _check(st, "gdn2_recurrent_update")
    return o


def gdn2_fg2_inputs(q, k, beta, q_out, k_out, b_out, w_out, *, stream=None):
    """FG^2-GDN inputs for the GDN-2 core (C ABI gdn2_fg2_inputs): writes q_out, k_out = sqrt(beta).k,
    b_out = 1, w_out = sqrt(beta), all per value head.

    q, k: [B, T, H_k, d] (or [B, H_k, d] for decode tokens); beta and the outputs: [B, T, H_v, d]
    (or [B, H_v, d]).
    """
    if q.dim() == 3:
        B, Hk, d = q.shape
        T, Hv = 1, beta.shape[1]
    else:
        B, T, Hk, d = q.shape
        Hv = beta.shape[2]
    st = lib.gdn2_fg2_inputs(_ptr(q), _ptr(k), _ptr(beta), _ptr(q_out), _ptr(k_out), _ptr(b_out), _ptr(w_out),
                             B, T, Hk, Hv, d, _dtype_code(q), _stream(stream))
    _check(st, "gdn2_fg2_inputs")
    return q_out, k_out, b_out, w_out


def fg2_inputs(q, k, beta, *, stream=None):
    """Returns (q_out, k_out, b_out, w_out) for running FG^2-GDN on the GDN-2 core (H_k = H_v)."""
    import torch

    outs = [torch.empty(beta.shape, dtype=q.dtype, device=q.device) for _ in range(4)]
    return gdn2_fg2_inputs(q, k, beta, *outs, stream=stream)


def gdn2_mixer_prologue(xq, xk, xv, conv_q, conv_k, conv_v, ag, ab, aw, q, k, v, g, b, w, states=None, *,
                        neg_eigval=False, stream=None):
    """ShortConv + L2 norm + gate activations (C ABI gdn2_mixer_prologue). Shapes as the core's
    inputs ([B, T, H, d], or [B, H, d] for one decode token); conv weights fp32 [H * d, 4];
    `states`: None or (state_q, state_k, state_v) fp32 [B, 3, H * d] tensors (each may be None),
    updated in place."""
    if xq.dim() == 3:
        B, Hk, dk = xq.shape
        T, Hv, dv = 1, xv.shape[1], xv.shape[2]
    else:
        B, T, Hk, dk = xq.shape
        Hv, dv = xv.shape[2], xv.shape[3]
    sq, sk, sv = states if states is not None else (None, None, None)
    st = lib.gdn2_mixer_prologue(*(_ptr(t) for t in (xq, xk, xv, conv_q, conv_k, conv_v, ag, ab, aw, sq, sk, sv,
                                                    q, k, v, g, b, w)),
                                 B, T, Hk, Hv, dk, dv, int(bool(neg_eigval)), _dtype_code(xq), _stream(stream))
    _check(st, "gdn2_mixer_prologue")
    return q, k, v, g, b, w


def gdn2_mixer_epilogue(o, z, weight, y, *, eps=1e-5, stream=None):
    """Gated RMSNorm with a SiLU gate (C ABI gdn2_mixer_epilogue); o, z, y: [B, T, H_v, d_v] (or
    [B, H_v, d_v]); weight: fp32 [d_v]."""
    if o.dim() == 3:
        B, Hv, dv = o.shape
        T = 1
    else:
        B, T, Hv, dv = o.shape
    st = lib.gdn2_mixer_epilogue(_ptr(o), _ptr(z), _ptr(weight), float(eps), _ptr(y), B, T, Hv, dv,
                                 _dtype_code(o), _stream(stream))
    _check(st, "gdn2_mixer_epilogue")
    return y


def gdn2_backward(q, k, v, g, b, w, d_o, dq, dk, dv, dg, db, dw, initial_state=None, d_final_state=None,
                  d_initial_state=None, *, scale=1.0, workspace=None, stream=None, recurrent=False):
    """Gradients of the core (C ABI gdn2_backward, or gdn2_backward_recurrent when `recurrent`);
    writes dq, dk, dv, dg, db, dw and, if given, d_initial_state. Shapes as gdn2_chunk_fwd's
    inputs; states fp32 [B, H_v, d_k, d_v]."""
    import torch

    B, T, Hk, dk_ = q.shape
    Hv, dv_ = v.shape[2], v.shape[3]
    dt = _dtype_code(q)
    size_fn = lib.gdn2_backward_recurrent_workspace_size if recurrent else lib.gdn2_backward_workspace_size
    fn = lib.gdn2_backward_recurrent if recurrent else lib.gdn2_backward
    need = size_fn(B, T, Hk, Hv, dk_, dv_, dt)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = fn(*(_ptr(t) for t in (q, k, v, g, b, w, initial_state, d_o, d_final_state, dq, dk, dv, dg, db, dw,
                                d_initial_state)),
            B, T, Hk, Hv, dk_, dv_, float(scale), dt, _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "gdn2_backward_recurrent" if recurrent else "gdn2_backward")
    return dq, dk, dv, dg, db, dw


def backward(q, k, v, g, b, w, d_o, initial_state=None, d_final_state=None, *, scale=1.0, stream=None,
             recurrent=False):
    """Returns (dq, dk, dv, dg, db, dw, d_initial_state)."""
    import torch

    outs = [torch.empty_like(t) for t in (q, k, v, g, b, w)]
    B, Hv, dk_, dv_ = q.shape[0], v.shape[2], q.shape[3], v.shape[3]
    ds0 = torch.empty((B, Hv, dk_, dv_), dtype=torch.float32, device=q.device)
    gdn2_backward(q, k, v, g, b, w, d_o, *outs, initial_state, d_final_state, ds0, scale=scale, stream=stream,
                  recurrent=recurrent)
    return (*outs, ds0)


def gdn2_last_device_status(stream=None) -> int:
    return lib.gdn2_last_device_status(_stream(stream))


def gdn2_set_wait_limit(ns: int) -> None:
    lib.gdn2_set_wait_limit(int(ns))


def gdn2_selftest_umma(case_id: int, soft: int, a, b, d, stream=None):
    _check(lib.gdn2_selftest_umma(case_id, soft, _ptr(a), _ptr(b), _ptr(d), _stream(stream)),
           "gdn2_selftest_umma")
    return d


# ---- convenience wrappers that allocate outputs (torch is used for memory only) -------------------

def chunk_fwd(q, k, v, g, b, w, initial_state=None, *, output_final_state=True, C=64, scale=1.0,
              path="auto", workspace=None, stream=None):
    """Returns (o, final_state or None)."""
    import torch

    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    o = torch.empty((B, T, Hv, dv), dtype=q.dtype, device=q.device)
    fs = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=q.device) if output_final_state else None
    return gdn2_chunk_fwd(q, k, v, g, b, w, o, initial_state, fs, C=C, scale=scale, workspace=workspace,
                          path=path, stream=stream)


def recurrent_step(q, k, v, g, b, w, state, *, scale=1.0, stream=None):
    """Returns o; `state` is updated in place."""
    import torch

    o = torch.empty(v.shape, dtype=q.dtype, device=q.device)
    return gdn2_recurrent_step(q, k, v, g, b, w, state, o, scale=scale, stream=stream)


def gdn2_mixer_decode_step(xq, xk, xv, conv_q, conv_k, conv_v, ag, ab, aw, state, z, weight, y, *,
                           states=(None, None, None), eps=1e-5, neg_eigval=False, scale=1.0, stream=None):
    """One decode token of the whole mixer (C ABI gdn2_mixer_decode_step): conv + L2 norm + gates,
    the recurrent update of `state` (in place) and the gated RMSNorm into `y`.

    xq, xk: [B, H_k, d_k]; xv, z, y: [B, H_v, d_v]; ag, ab: [B, H_v, d_k]; aw: [B, H_v, d_v] (one dtype);
    conv_*: float32 [channels, 4]; states: float32 conv states [B, 3, channels] or None (updated in
    place); state: float32 [B, H_v, d_k, d_v]; weight: float32 [d_v].
    """
    B, Hk, dk = xq.shape
    Hv, dv = xv.shape[1], xv.shape[2]
    sq, sk, sv = states
    st = lib.gdn2_mixer_decode_step(_ptr(xq), _ptr(xk), _ptr(xv), _ptr(conv_q), _ptr(conv_k), _ptr(conv_v),
                                    _ptr(ag), _ptr(ab), _ptr(aw), _ptr(sq), _ptr(sk), _ptr(sv), _ptr(state),
                                    _ptr(z), _ptr(weight), float(eps), _ptr(y), B, Hk, Hv, dk, dv,
                                    int(bool(neg_eigval)), float(scale), _dtype_code(xq), _stream(stream))
    _check(st, "gdn2_mixer_decode_step")
    return y


# ---- selective state-space mixer ------------------------------------------------------------------------
# A call here costs as much host time as many of the kernels run for, so arguments are checked and marshalled
# in one pass, pointers go to ctypes as integers, and workspace sizes are looked up by the call's sizes and device (they
# depend on its number of SMs).

@functools.lru_cache(maxsize=4096)
def _size_of(fn, dev, *sizes) -> int:
    return getattr(lib, fn)(*sizes)


def _device(t) -> int:
    """The index of the tensor's device, which has to be the current one: kernels are launched there."""
    import torch

    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must live on a CUDA device")
    if dev != torch._C._cuda_getDevice():
        raise ValueError("tensors must live on the current CUDA device")
    return dev


def _raw_stream(stream, dev):
    import torch

    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _on_stream(call):
    """`call` with what it allocates, workspace and results, from the memory of the stream that it runs on: that of its
    `stream` argument where one is given. The workspace is let go of when the call returns, with its kernels still to run;
    only work behind them may have that memory next, and their results lie in none that other streams still work on.
    Results are marked as in use by the caller's stream too. (To order inputs and results between streams is the caller's.)"""
    @functools.wraps(call)
    def run(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        import torch

        caller = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            got = call(*args, **kw)
        for t in got if isinstance(got, tuple) else (got,):
            if t is not None:
                t.record_stream(caller)
        return got

    run.plain = call  # for a call within a call
    return run


def _dense(t, dtype, shape, name, dev):
    """Pointer of a contiguous tensor of this dtype and shape on device `dev`; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: all tensors must live on the same CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, dtype, shape, tail, name, dev):
    """(pointer, row stride) of a token tensor [..., *tail]: each row's last `tail` dimensions are dense, the rows lie
    one stride apart (a slice of a wider row is fine)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: all token tensors share one dtype, {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: all tensors must live on the same CUDA device")
    width = shape[-1] if tail == 1 else shape[-1] * shape[-2]
    if t.is_contiguous():
        return t.data_ptr(), width
    stride = t.stride()
    dense = 1
    for i in range(len(shape) - 1, len(shape) - 1 - tail, -1):
        if shape[i] != 1 and stride[i] != dense:
            raise ValueError(f"{name}: the dimensions within a row must be dense")
        dense *= shape[i]
    ld = reach = None
    for i in range(len(shape) - 1 - tail, -1, -1):
        if shape[i] == 1:
            continue
        if ld is None:
            ld = reach = stride[i]
        elif stride[i] != reach:
            raise ValueError(f"{name}: rows must lie one stride apart")
        reach *= shape[i]
    return t.data_ptr(), width if ld is None else ld


def _lead(t, tail, offsets, dev):
    """Leading dimensions, B, T and the offsets' pointer of a call whose token tensors are [B, T, ...], or [T, ...] with
    offsets."""
    import torch

    lead = tuple(t.shape[:-tail])
    if offsets is None:
        if len(lead) != 2:
            raise ValueError("token tensors are [B, T, ...] (or [T, ...] with offsets)")
        return lead, lead[0], lead[1], None
    if len(lead) != 1:
        raise ValueError("with offsets, token tensors are [T, ...]")
    if offsets.dtype is not torch.int32 or offsets.dim() != 1 or offsets.shape[0] < 1:
        raise TypeError("offsets is an int32 tensor of one entry more than sequences")
    return lead, offsets.shape[0] - 1, lead[0], _dense(offsets, torch.int32, offsets.shape, "offsets", dev)


def _workspace(need, like, given, dev):
    """(tensor, pointer, bytes) of a call's workspace, allocated when none is given and one is needed."""
    import torch

    if given is None:
        if not need:
            return None, None, 0
        given = torch.empty(need, dtype=torch.uint8, device=like.device)
    return given, _dense(given, torch.uint8, given.shape, "workspace", dev), given.shape[0]


def _prologue(xbc, delta, conv_weight, conv_bias, a, delta_bias, conv_state, offsets, silu, stream, outs):
    import torch

    dev = _device(xbc)
    lead, B, T, off = _lead(xbc, 1, offsets, dev)
    ch, H, dtype, f32 = xbc.shape[-1], delta.shape[-1], xbc.dtype, torch.float32
    wide, narrow = (*lead, ch), (*lead, H)
    px, lx = _rows(xbc, dtype, wide, 1, "xbc", dev)
    pd, ld = _rows(delta, dtype, narrow, 1, "delta", dev)
    if outs is None:
        at = xbc.device
        outs = (torch.empty(wide, dtype=dtype, device=at), torch.empty(narrow, dtype=dtype, device=at),
                torch.empty(narrow, dtype=dtype, device=at))
        ptrs = [t.data_ptr() for t in outs]
    else:
        ptrs = [_dense(t, dtype, s, n, dev) for t, s, n in zip(outs, (wide, narrow, narrow), ("u", "step", "g"))]
    _check(lib.gdn2_ssm_prologue(px, lx, pd, ld, _dense(conv_weight, f32, (ch, 4), "conv_weight", dev),
                                 _dense(conv_bias, f32, (ch,), "conv_bias", dev), _dense(a, f32, (H,), "a", dev),
                                 _dense(delta_bias, f32, (H,), "delta_bias", dev), _dense(conv_state, f32, (B, 3, ch), "conv_state", dev),
                                 off, *ptrs, B, T, ch, H, 1 if silu else 0, _dtype_code(xbc), _raw_stream(stream, dev)),
           "gdn2_ssm_prologue")
    return outs


def gdn2_ssm_prologue(xbc, delta, conv_weight, conv_bias, a, delta_bias, u, step, g, conv_state=None, offsets=None, *,
                      silu=True, stream=None):
    """Causal depthwise convolution (width 4) and gates of the selective state-space mixer (C ABI
    gdn2_ssm_prologue): u = silu(conv(xbc) + conv_bias), step = softplus(delta + delta_bias), g = a * step.

    xbc, u: [B, T, channels]; delta, step, g: [B, T, H]; conv_weight: float32 [channels, 4]; conv_bias: float32
    [channels] or None; a, delta_bias: float32 [H]; conv_state: float32 [B, 3, channels], replaced in place, or None.
    With offsets (int32 [B + 1], on the device) the sequences are packed and token tensors are [T, ...]. xbc and delta
    may be slices of wider rows.
    """
    return _prologue(xbc, delta, conv_weight, conv_bias, a, delta_bias, conv_state, offsets, silu, stream, (u, step, g))


@_on_stream
def ssm_prologue(xbc, delta, conv_weight, conv_bias, a, delta_bias, conv_state=None, offsets=None, *, silu=True, stream=None):
    """Returns (u, step, g); conv_state, if given, is updated in place."""
    return _prologue(xbc, delta, conv_weight, conv_bias, a, delta_bias, conv_state, offsets, silu, stream, None)


@_on_stream
def gdn2_ssm_prologue_backward(xbc, delta, conv_weight, conv_bias, a, delta_bias, du, dstep, dg, dxbc, ddelta, dconv_weight,
                               dconv_bias, da, ddelta_bias, offsets=None, *, silu=True, workspace=None, stream=None):
    """Gradients of gdn2_ssm_prologue from zero convolution states (C ABI gdn2_ssm_prologue_backward); writes dxbc,
    ddelta (token dtype; may be slices of wider rows) and the float32 parameter gradients (dconv_bias may be None)."""
    import torch

    dev = _device(xbc)
    lead, B, T, off = _lead(xbc, 1, offsets, dev)
    ch, H, dtype, f32 = xbc.shape[-1], delta.shape[-1], xbc.dtype, torch.float32
    wide, narrow, dt = (*lead, ch), (*lead, H), _dtype_code(xbc)
    ws, pw, nw = _workspace(_size_of("gdn2_ssm_prologue_backward_workspace_size", dev, B, T, ch, H, int(off is not None), dt), xbc, workspace, dev)
    _check(lib.gdn2_ssm_prologue_backward(
        *_rows(xbc, dtype, wide, 1, "xbc", dev), *_rows(delta, dtype, narrow, 1, "delta", dev),
        _dense(conv_weight, f32, (ch, 4), "conv_weight", dev), _dense(conv_bias, f32, (ch,), "conv_bias", dev), _dense(a, f32, (H,), "a", dev),
        _dense(delta_bias, f32, (H,), "delta_bias", dev), off, *_rows(du, dtype, wide, 1, "du", dev), _dense(dstep, dtype, narrow, "dstep", dev),
        _dense(dg, dtype, narrow, "dg", dev), *_rows(dxbc, dtype, wide, 1, "dxbc", dev), *_rows(ddelta, dtype, narrow, 1, "ddelta", dev),
        _dense(dconv_weight, f32, (ch, 4), "dconv_weight", dev), _dense(dconv_bias, f32, (ch,), "dconv_bias", dev), _dense(da, f32, (H,), "da", dev),
        _dense(ddelta_bias, f32, (H,), "ddelta_bias", dev), B, T, ch, H, 1 if silu else 0, dt, pw, nw, _raw_stream(stream, dev)),
        "gdn2_ssm_prologue_backward")
    return dxbc, ddelta, dconv_weight, dconv_bias, da, ddelta_bias


@_on_stream
def ssm_prologue_backward(xbc, delta, conv_weight, conv_bias, a, delta_bias, du, dstep, dg, offsets=None, *, silu=True,
                          stream=None):
    """Returns (dxbc, ddelta, dconv_weight, dconv_bias or None, da, ddelta_bias)."""
    import torch

    dev = xbc.device
    new = lambda t: torch.empty(t.shape, dtype=t.dtype, device=dev)
    return gdn2_ssm_prologue_backward.plain(xbc, delta, conv_weight, conv_bias, a, delta_bias, du, dstep, dg, new(xbc), new(delta),
                                            new(conv_weight), new(conv_bias) if conv_bias is not None else None, new(a),
                                            new(delta_bias), offsets, silu=silu, stream=stream)


def _scan(x, step, g, bm, cm, d, initial_state, final_state, offsets, path, workspace, stream, y, want_state):
    import torch

    dev = _device(x)
    lead, B, T, off = _lead(x, 2, offsets, dev)
    H, P = x.shape[-2:]
    G, N = bm.shape[-2:]
    dtype, f32, dt, pth = x.dtype, torch.float32, _dtype_code(x), PATHS[path]
    full, heads, keys, state = (*lead, H, P), (*lead, H), (*lead, G, N), (B, H, N, P)
    rx = _rows(x, dtype, full, 2, "x", dev)
    if y is None:
        y = torch.empty(full, dtype=dtype, device=x.device)
        py = y.data_ptr()
    else:
        py = _dense(y, dtype, full, "y", dev)
    if want_state:
        final_state = torch.empty(state, dtype=f32, device=x.device)
    ws, pw, nw = _workspace(_size_of("gdn2_ssm_chunk_fwd_workspace_size", dev, pth, B, T, H, G, P, N, int(off is not None), dt), x, workspace, dev)
    _check(lib.gdn2_ssm_chunk_fwd(
        pth, *rx, _dense(step, dtype, heads, "step", dev), _dense(g, dtype, heads, "g", dev), *_rows(bm, dtype, keys, 2, "bm", dev),
        *_rows(cm, dtype, keys, 2, "cm", dev), _dense(d, f32, (H,), "d", dev), _dense(initial_state, f32, state, "initial_state", dev),
        _dense(final_state, f32, state, "final_state", dev), off, py, B, T, H, G, P, N, dt, pw, nw, _raw_stream(stream, dev)),
        "gdn2_ssm_chunk_fwd")
    return y, final_state


@_on_stream
def gdn2_ssm_chunk_fwd(x, step, g, bm, cm, y, d=None, initial_state=None, final_state=None, offsets=None, *, path="auto",
                       workspace=None, stream=None):
    """Selective state-space scan (C ABI gdn2_ssm_chunk_fwd): per head H_t = e^{g_t} H_{t-1} + step_t B_t x_t^T,
    y_t = H_t^T C_t + d x_t; writes y and, if given, final_state.

    x, y: [B, T, H, P]; step, g: [B, T, H]; bm, cm: [B, T, G, N]; d: float32 [H] or None; states: float32
    [B, H, N, P]. With offsets (int32 [B + 1], on the device) the sequences are packed and token tensors are [T, ...].
    x, bm and cm may be slices of wider rows.
    """
    return _scan(x, step, g, bm, cm, d, initial_state, final_state, offsets, path, workspace, stream, y, False)


@_on_stream
def ssm_chunk_fwd(x, step, g, bm, cm, d=None, initial_state=None, offsets=None, *, output_final_state=True, path="auto",
                  workspace=None, stream=None):
    """Returns (y, final_state or None)."""
    return _scan(x, step, g, bm, cm, d, initial_state, None, offsets, path, workspace, stream, None, output_final_state)


def _scan_grad(x, step, g, bm, cm, d_y, d, initial_state, d_final_state, offsets, path, workspace, stream, outs):
    import torch

    dev = _device(x)
    lead, B, T, off = _lead(x, 2, offsets, dev)
    H, P = x.shape[-2:]
    G, N = bm.shape[-2:]
    dtype, f32, dt, pth = x.dtype, torch.float32, _dtype_code(x), PATHS[path]
    full, heads, keys, state = (*lead, H, P), (*lead, H), (*lead, G, N), (B, H, N, P)
    rx, rb, rc = _rows(x, dtype, full, 2, "x", dev), _rows(bm, dtype, keys, 2, "bm", dev), _rows(cm, dtype, keys, 2, "cm", dev)
    if outs is None:
        at, hp, gn = x.device, H * P, G * N
        ch = hp + 2 * gn
        row = torch.empty((*lead, ch), dtype=dtype, device=at)
        back = (ch,) if off is not None else (T * ch, ch)
        dx = row.as_strided(full, (*back, P, 1))
        dbm, dcm = row.as_strided(keys, (*back, N, 1), hp), row.as_strided(keys, (*back, N, 1), hp + gn)
        dstep, dg = torch.empty(heads, dtype=dtype, device=at), torch.empty(heads, dtype=dtype, device=at)
        dd = torch.empty((H,), dtype=f32, device=at) if d is not None else None
        ds0 = torch.empty(state, dtype=f32, device=at) if initial_state is not None else None
        outs = (dx, dstep, dg, dbm, dcm, dd, ds0)
        base, es = row.data_ptr(), row.element_size()
        ox, ob, oc = (base, ch), (base + es * hp, ch), (base + es * (hp + gn), ch)
    else:
        dx, dstep, dg, dbm, dcm, dd, ds0 = outs
        ox, ob, oc = _rows(dx, dtype, full, 2, "dx", dev), _rows(dbm, dtype, keys, 2, "dbm", dev), _rows(dcm, dtype, keys, 2, "dcm", dev)
    ws, pw, nw = _workspace(_size_of("gdn2_ssm_backward_workspace_size", dev, pth, B, T, H, G, P, N, int(off is not None), dt), x, workspace, dev)
    _check(lib.gdn2_ssm_backward(
        pth, *rx, _dense(step, dtype, heads, "step", dev), _dense(g, dtype, heads, "g", dev), *rb, *rc, _dense(d, f32, (H,), "d", dev),
        _dense(initial_state, f32, state, "initial_state", dev), *_rows(d_y, dtype, full, 2, "d_y", dev),
        _dense(d_final_state, f32, state, "d_final_state", dev), off, *ox, _dense(dstep, dtype, heads, "dstep", dev),
        _dense(dg, dtype, heads, "dg", dev), *ob, *oc, _dense(dd, f32, (H,), "dd", dev), _dense(ds0, f32, state, "d_initial_state", dev),
        B, T, H, G, P, N, dt, pw, nw, _raw_stream(stream, dev)), "gdn2_ssm_backward")
    return outs


@_on_stream
def gdn2_ssm_backward(x, step, g, bm, cm, d_y, dx, dstep, dg, dbm, dcm, dd=None, d=None, initial_state=None,
                      d_final_state=None, d_initial_state=None, offsets=None, *, path="auto", workspace=None, stream=None):
    """Gradients of gdn2_ssm_chunk_fwd (C ABI gdn2_ssm_backward); writes dx, dstep, dg, dbm, dcm (token dtype; dx, dbm
    and dcm may be slices of wider rows) and, if given, the float32 dd and d_initial_state."""
    return _scan_grad(x, step, g, bm, cm, d_y, d, initial_state, d_final_state, offsets, path, workspace, stream,
                      (dx, dstep, dg, dbm, dcm, dd, d_initial_state))


@_on_stream
def ssm_backward(x, step, g, bm, cm, d_y, d=None, initial_state=None, d_final_state=None, offsets=None, *, path="auto",
                 workspace=None, stream=None):
    """Returns (dx, dstep, dg, dbm, dcm, dd, d_initial_state); dd is None without d, d_initial_state without initial_state.
    dx, dbm and dcm are slices of one row [..., H * P + 2 * G * N], the layout of the prologue's u and du."""
    return _scan_grad(x, step, g, bm, cm, d_y, d, initial_state, d_final_state, offsets, path, workspace, stream, None)


@_on_stream
def gdn2_ssm_decode_step(xbc, delta, conv_weight, conv_bias, a, delta_bias, d, conv_state, state, y, slots=None, *, stream=None):
    """One token of the selective state-space mixer between its projections (C ABI gdn2_ssm_decode_step): convolution
    with SiLU, gates, state update and readout in one launch.

    xbc: [B, channels] with channels = H P + 2 G N (x, B, C side by side); delta: [B, H] (both may be slices of wider
    rows); y: [B, H, P]; conv_state: float32 [B, 3, channels]; state: float32 or bfloat16 [B, H, N, P], both updated in
    place; with slots (int32 [B]) they are pools [n_slots, ...] and a slot out of range leaves its row untouched.
    """
    import torch

    dev = _device(xbc)
    B, ch = xbc.shape
    rows, H, N, P = state.shape
    G = (ch - H * P) // (2 * N)
    if ch != H * P + 2 * G * N or G < 1:
        raise ValueError("xbc holds H * P + 2 * G * N channels")
    if slots is None and rows != B:
        raise ValueError("without slots, the states have one row per sequence")
    dtype, f32 = xbc.dtype, torch.float32
    if y is None:
        y = torch.empty((B, H, P), dtype=dtype, device=xbc.device)
    _check(lib.gdn2_ssm_decode_step(
        *_rows(xbc, dtype, (B, ch), 1, "xbc", dev), *_rows(delta, dtype, (B, H), 1, "delta", dev), _dense(conv_weight, f32, (ch, 4), "conv_weight", dev),
        _dense(conv_bias, f32, (ch,), "conv_bias", dev), _dense(a, f32, (H,), "a", dev), _dense(delta_bias, f32, (H,), "delta_bias", dev),
        _dense(d, f32, (H,), "d", dev), _dense(conv_state, f32, (rows, 3, ch), "conv_state", dev), _dense(state, state.dtype, state.shape, "state", dev),
        _dtype_code(state), _dense(slots, torch.int32, (B,), "slots", dev), rows if slots is not None else 0,
        _dense(y, dtype, (B, H, P), "y", dev), B, H, G, P, N, _dtype_code(xbc), _raw_stream(stream, dev)), "gdn2_ssm_decode_step")
    return y


@_on_stream
def ssm_decode_step(xbc, delta, conv_weight, conv_bias, a, delta_bias, d, conv_state, state, slots=None, *, stream=None):
    """Returns y [B, H, P]; conv_state and state are updated in place. Rows of inactive slots are left unwritten."""
    return gdn2_ssm_decode_step.plain(xbc, delta, conv_weight, conv_bias, a, delta_bias, d, conv_state, state, None, slots, stream=stream)


def gdn2_block_norm(x, z, post_weight, residual, scale, pre_weight, r, n, *, groups=1, eps=1e-5, stream=None):
    """The residual stream around a block (C ABI gdn2_block_norm): p = post_weight * t / rms_group(t) with
    t = x silu(z), r = residual + scale p, n = pre_weight * r / rms(r). z, post_weight, residual, scale and pre_weight
    may each be None; r may be None when n is wanted alone. x, z, residual, r, n: [..., d]; weights: float32 [d]."""
    import torch

    dev = _device(x)
    shape, dtype, f32 = x.shape, x.dtype, torch.float32
    dim = shape[-1]
    vec = (dim,)
    _check(lib.gdn2_block_norm(
        _dense(x, dtype, shape, "x", dev), _dense(z, dtype, shape, "z", dev), _dense(post_weight, f32, vec, "post_weight", dev),
        _dense(residual, dtype, shape, "residual", dev), _dense(scale, f32, vec, "scale", dev), _dense(pre_weight, f32, vec, "pre_weight", dev),
        _dense(r, dtype, shape, "r", dev), _dense(n, dtype, shape, "n", dev), x.numel() // dim if dim else 0, dim, groups, float(eps),
        _dtype_code(x), _raw_stream(stream, dev)), "gdn2_block_norm")
    return r, n


@_on_stream
def block_norm(x, z=None, post_weight=None, residual=None, scale=None, pre_weight=None, *, groups=1, eps=1e-5, stream=None):
    """Returns (r, n): r is None when there is a norm before the next block but no residual to carry on; n is None
    without pre_weight."""
    import torch

    r = torch.empty_like(x) if residual is not None or pre_weight is None else None
    n = torch.empty_like(x) if pre_weight is not None else None
    return gdn2_block_norm(x, z, post_weight, residual, scale, pre_weight, r, n, groups=groups, eps=eps, stream=stream)


@_on_stream
def gdn2_block_norm_backward(x, z, post_weight, residual, scale, pre_weight, d_r, d_n, dx, dz, dpost_weight, dresidual, dscale,
                             dpre_weight, *, groups=1, eps=1e-5, workspace=None, stream=None):
    """Gradients of gdn2_block_norm (C ABI gdn2_block_norm_backward) given those of r (d_r, or None) and n (d_n, with
    pre_weight): one output for each input given; dresidual may be None."""
    import torch

    dev = _device(x)
    shape, dtype, f32 = x.shape, x.dtype, torch.float32
    dim = shape[-1]
    rows, vec = x.numel() // dim if dim else 0, (dim,)
    ws, pw, nw = _workspace(_size_of("gdn2_block_norm_backward_workspace_size", dev, rows, dim), x, workspace, dev)
    tok = lambda t, k: _dense(t, dtype, shape, k, dev)
    par = lambda t, k: _dense(t, f32, vec, k, dev)
    _check(lib.gdn2_block_norm_backward(
        tok(x, "x"), tok(z, "z"), par(post_weight, "post_weight"), tok(residual, "residual"), par(scale, "scale"),
        par(pre_weight, "pre_weight"), tok(d_r, "d_r"), tok(d_n, "d_n"), tok(dx, "dx"), tok(dz, "dz"),
        par(dpost_weight, "dpost_weight"), tok(dresidual, "dresidual"), par(dscale, "dscale"), par(dpre_weight, "dpre_weight"),
        rows, dim, groups, float(eps), _dtype_code(x), pw, nw, _raw_stream(stream, dev)), "gdn2_block_norm_backward")
    return dx, dz, dpost_weight, dresidual, dscale, dpre_weight


@_on_stream
def block_norm_backward(x, z=None, post_weight=None, residual=None, scale=None, pre_weight=None, d_r=None, d_n=None, *,
                        groups=1, eps=1e-5, stream=None):
    """Returns (dx, dz, dpost_weight, dresidual, dscale, dpre_weight), None for inputs not given."""
    import torch

    new = lambda t: torch.empty_like(t) if t is not None else None
    return gdn2_block_norm_backward.plain(x, z, post_weight, residual, scale, pre_weight, d_r, d_n, new(x), new(z), new(post_weight),
                                          new(residual), new(scale), new(pre_weight), groups=groups, eps=eps, stream=stream)


# ---- attention layers: norm and rotation, a cache in pages, attention over it ---------------------------------------

def _turned(q, k, q_weight, k_weight, inv_freq, positions, offsets, dev):
    """What the prologue's calls share: leading dimensions, sizes and the pointers of the tensors that all of them take."""
    import torch

    lead, B, T, off = _lead(q, 2, offsets, dev)
    (Hq, d), Hkv, f32 = q.shape[-2:], k.shape[-2], torch.float32
    if inv_freq is not None and inv_freq.dim() != 1:
        raise ValueError("inv_freq holds one frequency for each pair of rotated elements")
    rot = 2 * inv_freq.shape[0] if inv_freq is not None else 0
    params = (_dense(q_weight, f32, (d,), "q_weight", dev), _dense(k_weight, f32, (d,), "k_weight", dev),
              _dense(inv_freq, f32, (rot // 2,), "inv_freq", dev), _dense(positions, torch.int32, lead, "positions", dev), off)
    heads, keys = (*lead, Hq, d), (*lead, Hkv, d)
    return (*_rows(q, q.dtype, heads, 2, "q", dev), *_rows(k, q.dtype, keys, 2, "k", dev)), params, heads, keys, (B, T, Hq, Hkv, d, rot)


@_on_stream
def gdn2_attn_prologue(q, k, q_weight, k_weight, inv_freq, q_out, k_out, positions=None, offsets=None, *, interleaved=False, eps=1e-6,
                       stream=None):
    """RMS norm of each head of q and k and rotation by position (C ABI gdn2_attn_prologue); writes q_out and k_out.

    q, q_out: [B, T, H_q, d]; k, k_out: [B, T, H_kv, d]; weights: float32 [d] or None (no norm); inv_freq: float32, one for each pair
    of rotated elements, or None (no rotation); positions: int32 [B, T] or None (the index in the sequence). With offsets (int32
    [B + 1], on the device) the sequences are packed and token tensors are [T, ...]. q and k may be slices of wider rows.
    """
    dev = _device(q)
    rows, params, heads, keys, sizes = _turned(q, k, q_weight, k_weight, inv_freq, positions, offsets, dev)
    _check(lib.gdn2_attn_prologue(*rows, *params, _dense(q_out, q.dtype, heads, "q_out", dev), _dense(k_out, q.dtype, keys, "k_out", dev),
                                  *sizes, int(bool(interleaved)), float(eps), _dtype_code(q), _raw_stream(stream, dev)), "gdn2_attn_prologue")
    return q_out, k_out


@_on_stream
def attn_prologue(q, k, q_weight=None, k_weight=None, inv_freq=None, positions=None, offsets=None, *, interleaved=False, eps=1e-6,
                  stream=None):
    """Returns (q, k), normalised and rotated."""
    import torch

    return gdn2_attn_prologue.plain(q, k, q_weight, k_weight, inv_freq, torch.empty(q.shape, dtype=q.dtype, device=q.device),
                                    torch.empty(k.shape, dtype=q.dtype, device=q.device), positions, offsets, interleaved=interleaved,
                                    eps=eps, stream=stream)


def _cache(table, lengths, slots, B, dev):
    """Pointers and sizes of a cache's table, lengths and slots for a call of B rows."""
    import torch

    if table.dim() != 2:
        raise ValueError("table is [n_slots, max_pages]")
    rows = table.shape[0]
    if slots is None and rows != B:
        raise ValueError("without slots, the table has one row per sequence")
    i32 = torch.int32
    return (_dense(table, i32, table.shape, "table", dev), _dense(lengths, i32, (rows,), "lengths", dev),
            _dense(slots, i32, (B,), "slots", dev)), rows, table.shape[1]


def _pool(pages, dtype, Hkv, d, name, dev, like=None):
    """Pointer of a layer's pool [n_pages, H_kv, page, d]."""
    if pages.dim() != 4 or pages.shape[1] != Hkv or pages.shape[3] != d or (like is not None and pages.shape != like.shape):
        raise ValueError(f"{name} is [n_pages, H_kv, page, d], alike for keys and values")
    return _dense(pages, dtype, pages.shape, name, dev)


@_on_stream
def gdn2_attn_prologue_paged(q, k, v, k_pages, v_pages, table, lengths, q_out, slots=None, q_weight=None, k_weight=None, inv_freq=None,
                             positions=None, offsets=None, *, interleaved=False, eps=1e-6, stream=None):
    """The prologue for serving (C ABI gdn2_attn_prologue_paged): writes q_out, and k (normalised and rotated) and v to their places in
    the cache.

    q, k, v: as for gdn2_attn_prologue; k_pages, v_pages: [n_pages, H_kv, page, d]; table: int32 [n_slots, max_pages]; lengths: int32
    [n_slots], the call's tokens among them; slots: int32 [B] or None. positions, if given, are for the angles alone.
    """
    dev = _device(q)
    rows, params, heads, keys, sizes = _turned(q, k, q_weight, k_weight, inv_freq, positions, offsets, dev)
    B, _, _, Hkv, d, _ = sizes
    where, n_slots, wide = _cache(table, lengths, slots, B, dev)
    if q_out is None:
        import torch

        q_out = torch.empty(heads, dtype=q.dtype, device=q.device)
    _check(lib.gdn2_attn_prologue_paged(
        *rows, *_rows(v, q.dtype, keys, 2, "v", dev), *params, _dense(q_out, q.dtype, heads, "q_out", dev),
        _pool(k_pages, q.dtype, Hkv, d, "k_pages", dev), _pool(v_pages, q.dtype, Hkv, d, "v_pages", dev, k_pages), *where, n_slots,
        k_pages.shape[0], wide, k_pages.shape[2], *sizes, int(bool(interleaved)), float(eps), _dtype_code(q), _raw_stream(stream, dev)),
        "gdn2_attn_prologue_paged")
    return q_out


@_on_stream
def attn_prologue_paged(q, k, v, k_pages, v_pages, table, lengths, slots=None, q_weight=None, k_weight=None, inv_freq=None, positions=None,
                        offsets=None, *, interleaved=False, eps=1e-6, stream=None):
    """Returns q, normalised and rotated; k_pages and v_pages are updated in place. Rows of inactive slots are left unwritten."""
    return gdn2_attn_prologue_paged.plain(q, k, v, k_pages, v_pages, table, lengths, None, slots, q_weight, k_weight, inv_freq, positions,
                                          offsets, interleaved=interleaved, eps=eps, stream=stream)


@_on_stream
def gdn2_attn_prologue_backward(q, k, dq_out, dk_out, q_weight, k_weight, inv_freq, dq, dk, dq_weight, dk_weight, positions=None,
                                offsets=None, *, interleaved=False, eps=1e-6, workspace=None, stream=None):
    """Gradients of gdn2_attn_prologue (C ABI gdn2_attn_prologue_backward) given those of its outputs; writes dq and dk (may be slices of
    wider rows) and the float32 dq_weight and dk_weight, each with its weight."""
    import torch

    dev = _device(q)
    rows, params, heads, keys, sizes = _turned(q, k, q_weight, k_weight, inv_freq, positions, offsets, dev)
    B, T, _, _, d, _ = sizes
    need = _size_of("gdn2_attn_prologue_backward_workspace_size", dev, B, T, d, int(offsets is not None)) if dq_weight is not None or dk_weight is not None else 0
    ws, pw, nw = _workspace(need, q, workspace, dev)
    _check(lib.gdn2_attn_prologue_backward(
        *rows, *params, *_rows(dq_out, q.dtype, heads, 2, "dq_out", dev), *_rows(dk_out, q.dtype, keys, 2, "dk_out", dev),
        *_rows(dq, q.dtype, heads, 2, "dq", dev), *_rows(dk, q.dtype, keys, 2, "dk", dev),
        _dense(dq_weight, torch.float32, (d,), "dq_weight", dev), _dense(dk_weight, torch.float32, (d,), "dk_weight", dev), *sizes,
        int(bool(interleaved)), float(eps), _dtype_code(q), pw, nw, _raw_stream(stream, dev)), "gdn2_attn_prologue_backward")
    return dq, dk, dq_weight, dk_weight


@_on_stream
def attn_prologue_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, inv_freq=None, positions=None, offsets=None, *,
                           interleaved=False, eps=1e-6, stream=None):
    """Returns (dq, dk, dq_weight, dk_weight), the latter None without their weights."""
    import torch

    new = lambda t: torch.empty(t.shape, dtype=t.dtype, device=q.device) if t is not None else None
    return gdn2_attn_prologue_backward.plain(q, k, dq_out, dk_out, q_weight, k_weight, inv_freq, new(q), new(k), new(q_weight), new(k_weight),
                                             positions, offsets, interleaved=interleaved, eps=eps, stream=stream)


@_on_stream
def gdn2_attn_decode(q, k_pages, v_pages, table, lengths, o, slots=None, *, scale=None, window=0, workspace=None, stream=None):
    """Attention of the newest tokens of each row over its cache (C ABI gdn2_attn_decode); writes o.

    q, o: [B, N, H_q, d], or [B, H_q, d] for one token each (q may be a slice of wider rows); k_pages, v_pages: [n_pages, H_kv, page, d];
    table: int32 [n_slots, max_pages]; lengths: int32 [n_slots], these tokens among them; slots: int32 [B] or None. Token n sees the
    keys up to number lengths - N + n, with window > 0 the last `window` of them. scale: d ** -0.5 when None.
    """
    import torch

    dev = _device(q)
    if q.dim() not in (3, 4) or k_pages.dim() != 4:
        raise ValueError("q is [B, N, H_q, d] or [B, H_q, d], k_pages [n_pages, H_kv, page, d]")
    B, (Hq, d), N, Hkv = q.shape[0], q.shape[-2:], q.shape[1] if q.dim() == 4 else 1, k_pages.shape[1]
    where, n_slots, wide = _cache(table, lengths, slots, B, dev)
    dt = _dtype_code(q)
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    ws, pw, nw = _workspace(_size_of("gdn2_attn_decode_workspace_size", dev, B, N, Hq, Hkv, d, wide, k_pages.shape[2], dt), q, workspace, dev)
    _check(lib.gdn2_attn_decode(
        *_rows(q, q.dtype, q.shape, 2, "q", dev), _pool(k_pages, q.dtype, Hkv, d, "k_pages", dev),
        _pool(v_pages, q.dtype, Hkv, d, "v_pages", dev, k_pages), *where, n_slots, k_pages.shape[0], wide, k_pages.shape[2],
        _dense(o, q.dtype, q.shape, "o", dev), B, N, Hq, Hkv, d, float(d ** -0.5 if scale is None else scale),
        min(_int(window, "window", 0, 2 ** 62), 2 ** 31 - 1), dt, pw, nw,
        _raw_stream(stream, dev)), "gdn2_attn_decode")
    return o


@_on_stream
def attn_decode(q, k_pages, v_pages, table, lengths, slots=None, *, scale=None, window=0, stream=None):
    """Returns o, like q. Rows of inactive slots are left unwritten."""
    return gdn2_attn_decode.plain(q, k_pages, v_pages, table, lengths, None, slots, scale=scale, window=window, stream=stream)


def _pages(table, lengths, refs, dev):
    """Pointers and sizes of a cache's table, lengths and references."""
    import torch

    if table.dim() != 2 or refs.dim() != 1:
        raise ValueError("table is [n_slots, max_pages], refs [n_pages]")
    i32, (rows, wide), pages = torch.int32, table.shape, refs.shape[0]
    return (_dense(table, i32, table.shape, "table", dev), _dense(lengths, i32, (rows,), "lengths", dev),
            _dense(refs, i32, (pages,), "refs", dev)), rows, pages, wide


def _int(v, name, least, most):
    """v as an int in [least, most]: the C types would wrap what lies outside."""
    v = operator.index(v)
    if not least <= v <= most:
        raise ValueError(f"{name}: {least} to {most} expected, got {v}")
    return v


def _indices(t, name, dev, n=None):
    """Pointer of an int32 tensor [n] of row or page numbers."""
    import torch

    if t.dim() != 1:
        raise ValueError(f"{name} is an int32 tensor [n]")
    return _dense(t, torch.int32, (t.shape[0] if n is None else n,), name, dev)


def _active(t, dev, n, *inputs):
    """Pointer of the int32 tensor [n] that rows which take part are written to, apart from the call's own rows; None for None."""
    if t is None:
        return None
    if n and any(t.data_ptr() == i.data_ptr() for i in inputs):
        raise ValueError("active lies in memory of its own")
    return _indices(t, "active", dev, n)


@_on_stream
def pages_append(table, lengths, refs, slots, tokens, *, page, active=None, stream=None):
    """Room for more tokens behind rows `slots` (C ABI gdn2_pages_append, gdn2_pages_append_active): lengths grows by `tokens` (an int for every
    row, or int32 [n]) and the rows get the free pages that this takes, lowest first; table, lengths and refs are updated in place. slots are
    distinct. A row is shortened by lowering its length: its next tokens go to the pages that it keeps behind it.
    Returns ok: int32 [n], 0 where the row stays as it was (inactive, full, no pages left, or tokens that would get to a page of other rows too).
    active (int32 [n], beside slots): written with slots[i], or -1 where ok is 0: the slots of the step's other calls, which would else take such a
    row's newest tokens for the step's own and write over them."""
    import torch

    dev = _device(table)
    where, rows, pages, wide = _pages(table, lengths, refs, dev)
    n, each, counts = slots.shape[0], 0, None
    if isinstance(tokens, torch.Tensor):
        counts = _indices(tokens, "tokens", dev, n)
    else:
        each = _int(tokens, "tokens", 0, 2 ** 31 - 1)
    ok = torch.empty((n,), dtype=torch.int32, device=table.device)
    _check(lib.gdn2_pages_append_active(*where, _indices(slots, "slots", dev), counts, each, ok.data_ptr(), _active(active, dev, n, slots), n, rows,
                                        pages, wide, _int(page, "page", 1, 65536), _raw_stream(stream, dev)), "gdn2_pages_append")
    return ok


@_on_stream
def pages_fork(table, lengths, refs, src, dst, *, page, active=None, stream=None):
    """Rows `dst` (distinct) become rows like `src` (C ABI gdn2_pages_fork): dst rows are emptied, full pages shared, a last page that is not full
    gets a free page of its own; table, lengths and refs are updated in place. Returns (copy_from, copy_to, ok), int32 [n] each: what to copy in
    every layer's pools (pages_copy; -1 for nothing), and 0 where dst is left empty (inactive, or no pages left). active (int32 [n], beside
    dst): written with dst[i], or -1 where ok is 0 (gdn2_pages_fork_active): the slots of the calls behind it."""
    import torch

    dev = _device(table)
    where, rows, pages, wide = _pages(table, lengths, refs, dev)
    n = src.shape[0]
    copy_from, copy_to, ok = (torch.empty((n,), dtype=torch.int32, device=table.device) for _ in range(3))
    _check(lib.gdn2_pages_fork_active(*where, _indices(src, "src", dev), _indices(dst, "dst", dev, n), copy_from.data_ptr(), copy_to.data_ptr(),
                                      ok.data_ptr(), _active(active, dev, n, src, dst), n, rows, pages, wide, _int(page, "page", 1, 65536),
                                      _raw_stream(stream, dev)), "gdn2_pages_fork")
    return copy_from, copy_to, ok


@_on_stream
def pages_release(table, lengths, refs, slots, *, stream=None):
    """Empties rows `slots` (C ABI gdn2_pages_release): their pages are given back; table, lengths and refs are updated in place."""
    dev = _device(table)
    where, rows, pages, wide = _pages(table, lengths, refs, dev)
    _check(lib.gdn2_pages_release(*where, _indices(slots, "slots", dev), slots.shape[0], rows, pages, wide, _raw_stream(stream, dev)),
           "gdn2_pages_release")


@_on_stream
def pages_copy(pools, copy_from, copy_to, *, stream=None):
    """Copies rows copy_from[i] to rows copy_to[i] (int32 [n]; pairs with an index out of range are skipped) in each of `pools` (C ABI
    gdn2_pages_copy): a layer's pages, or the mixers' states by slot. Pools are contiguous, of any type, with equally many rows. The copy_to rows
    are distinct, and none is a copy_from row."""
    if not pools:
        return
    dev, rows, n = _device(pools[0]), pools[0].shape[0], copy_from.shape[0]
    ptrs, sizes, count = [], [], len(pools)
    for t in pools:
        shape = t.shape
        if shape[0] != rows:
            raise ValueError("pools have equally many rows")
        ptrs.append(_dense(t, t.dtype, shape, "pools", dev))
        sizes.append(t.nbytes // rows if rows else 0)
    _check(lib.gdn2_pages_copy((ctypes.c_void_p * count)(*ptrs), (ctypes.c_longlong * count)(*sizes), count, _indices(copy_from, "copy_from", dev),
                               _indices(copy_to, "copy_to", dev, n), n, rows, _raw_stream(stream, dev)), "gdn2_pages_copy")
