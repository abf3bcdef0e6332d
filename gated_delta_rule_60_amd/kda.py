"""Thin ctypes binding of libkda.so: the C ABI in include/kda.h, called with torch tensors.

Argument marshalling only -- every step of the computation runs in the HIP library.  The
functions keep the C names and raise ``KDAError`` for any status other than KDA_OK.  Loading
fails loudly when the built library is missing: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .build import lib_path

KDA_F32, KDA_BF16 = 0, 1
KDA_OK = 0
_DT = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}


class KDAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {kda_status_string(status)} ({status})")
        self.status = status


_lib = None


def load_library(path: Optional[str] = None):
    """Load libkda.so (default: the in-tree build).  Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libkda.so not found at {path}; build it first "
                           "(python -m gated_delta_rule_60_amd.build)")
    lib = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_version.argtypes = []
    lib.kda_version.restype = ctypes.c_int
    lib.kda_gate.argtypes = [vp, vp, ctypes.c_int, vp, ctypes.c_int, i64, i32, i32, f32, vp]
    lib.kda_gate.restype = ctypes.c_int
    lib.kda_chunk_fwd_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32, ctypes.c_int]
    lib.kda_chunk_fwd_workspace_size.restype = sz
    lib.kda_chunk_fwd.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp, vp,
                                  ctypes.c_int, i32, i64, i32, i32, i32, i32, i32, f32, vp, sz, vp]
    lib.kda_chunk_fwd.restype = ctypes.c_int
    lib.kda_chunk_fwd_gated.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp, ctypes.c_int, f32,
                                        vp, vp, vp, vp, ctypes.c_int, i32, i64, i32, i32, i32,
                                        i32, i32, f32, vp, sz, vp]
    lib.kda_chunk_fwd_gated.restype = ctypes.c_int
    lib.kda_chunk_fwd_gated_noalloc.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp,
                                                ctypes.c_int, f32, vp, vp, vp, vp, ctypes.c_int,
                                                i32, i64, i32, i32, i32, i32, i32, f32, vp]
    lib.kda_chunk_fwd_gated_noalloc.restype = ctypes.c_int
    lib.kda_chunk_fwd_checkpointed.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp, ctypes.c_int,
                                               f32, vp, vp, vp, vp, ctypes.c_int, i32, i64, i32,
                                               i32, i32, i32, i32, f32, vp, i32, i64, vp, sz, vp]
    lib.kda_chunk_fwd_checkpointed.restype = ctypes.c_int
    lib.kda_decode_step.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp,
                                    ctypes.c_int, i32, i32, i32, i32, f32, vp]
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_decode_verify.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp,
                                      ctypes.c_int, i32, i32, i32, i32, i32, f32, vp]
    lib.kda_decode_verify.restype = ctypes.c_int
    lib.kda_decode_commit.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp,
                                      i32, i32, i32, i32, i32, vp]
    lib.kda_decode_commit.restype = ctypes.c_int
    lib.kda_linear_chunk_workspace_size.argtypes = [i32, i64, i32, i32, i32, ctypes.c_int,
                                                    ctypes.c_int]
    lib.kda_linear_chunk_workspace_size.restype = sz
    lib.kda_linear_chunk_fwd.argtypes = [vp, vp, vp, ctypes.c_int, vp, vp, vp, vp, vp, ctypes.c_int,
                                         i32, i64, i32, i32, i32, i32, f32, vp, sz, vp]
    lib.kda_linear_chunk_fwd.restype = ctypes.c_int
    lib.kda_linear_chunk_bwd.argtypes = [vp, vp, vp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp,
                                         vp, i32, i64, i32, i32, i32, i32, f32, vp, sz, vp]
    lib.kda_linear_chunk_bwd.restype = ctypes.c_int
    lib.kda_linear_decode_step.argtypes = [vp, vp, vp, ctypes.c_int, vp, vp, vp, ctypes.c_int, i32,
                                           i32, i32, i32, f32, vp]
    lib.kda_linear_decode_step.restype = ctypes.c_int
    lib.kda_state_store.argtypes = [vp, vp, vp, ctypes.c_int, vp, i32, i32, i32, i32, i32, i32, vp]
    lib.kda_state_store.restype = ctypes.c_int
    lib.kda_state_load.argtypes = [vp, ctypes.c_int, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp]
    lib.kda_state_load.restype = ctypes.c_int
    ci = ctypes.c_int
    signatures = {
        "kda_conv_bwd_workspace_size": [i32, i64, i32, i32],
        "kda_conv_fwd": [vp, i64, ci, vp, vp, vp, vp, vp, vp, i64, i32, i64, i32, i32, i32, ci, vp],
        "kda_conv_bwd": [vp, i64, ci, vp, vp, vp, vp, vp, i64, vp, vp, i64, vp, vp, vp, i32, i64, i32, i32,
                         i32, ci, vp, sz, vp],
        "kda_conv_step": [vp, i64, ci, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, ci, vp],
        "kda_ssm_chunk_workspace_size": [i32, i64, i32, i32, i32, i32, ci, ci],
        "kda_ssm_chunk_fwd": [vp, i64, vp, i64, vp, i64, vp, i64, ci, vp, vp, vp, vp, vp, vp, vp, i64, ci,
                              i32, i64, i32, i32, i32, i32, i32, vp, sz, vp],
        "kda_ssm_chunk_bwd": [vp, i64, vp, i64, vp, i64, vp, i64, ci, vp, vp, vp, vp, vp, vp, i64, vp, vp,
                              i64, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32,
                              i32, vp, sz, vp],
        "kda_ssm_decode_step": [vp, i64, vp, i64, vp, i64, vp, i64, ci, vp, vp, vp, vp, vp, vp, i64, ci,
                                i32, i32, i32, i32, i32, i32, vp],
        "kda_slots_workspace_size": [i32, i32],
        "kda_slots_copy": [vp, vp, vp, i32, vp, vp, i32, i32, i32, vp],
        "kda_slots_retain": [vp, vp, i32, i32, vp],
        "kda_slots_release": [vp, vp, i32, i32, vp],
        "kda_slots_fork": [vp, vp, i32, vp, vp, vp, i32, i32, vp, sz, vp],
        "kda_slots_compact": [vp, vp, i32, vp, vp, i64, vp, i32, vp, sz, vp],
    }
    for name, argtypes in signatures.items():
        getattr(lib, name).argtypes = argtypes
        getattr(lib, name).restype = sz if name.endswith("_workspace_size") else ci
    if path == lib_path():
        _lib = lib
    return lib


EXPORTED = ["kda_status_string", "kda_version", "kda_gate", "kda_chunk_fwd_workspace_size",
            "kda_chunk_fwd", "kda_chunk_fwd_gated", "kda_chunk_fwd_gated_noalloc",
            "kda_chunk_fwd_checkpointed", "kda_decode_step", "kda_decode_verify",
            "kda_decode_commit", "kda_linear_chunk_workspace_size", "kda_linear_chunk_fwd",
            "kda_linear_chunk_bwd", "kda_linear_decode_step", "kda_state_store", "kda_state_load",
            "kda_conv_bwd_workspace_size", "kda_conv_fwd", "kda_conv_bwd", "kda_conv_step",
            "kda_ssm_chunk_workspace_size", "kda_ssm_chunk_fwd", "kda_ssm_chunk_bwd",
            "kda_ssm_decode_step", "kda_slots_workspace_size", "kda_slots_copy", "kda_slots_retain",
            "kda_slots_release", "kda_slots_fork", "kda_slots_compact"]

# Size of the library's static prefill workspace used by kda_chunk_fwd_gated_noalloc.
NOALLOC_SCRATCH_BYTES = 256 << 20


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libkda must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _dt(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)") from None


_FLOATS = (torch.float32, torch.bfloat16)


def _expect(fn: str, name: str, t, shape, dtypes=None):
    """Host-side argument check: t (None = absent) must be a contiguous tensor of the given
    shape (None entries match any size) and, when given, one of `dtypes`."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{fn}: {name} must be a torch.Tensor")
    if (dtypes is None or t.dtype in dtypes) and t.is_contiguous():
        size = t.shape
        if size == shape:
            return
        if len(size) == len(shape):
            for a, w in zip(size, shape):
                if w is not None and a != w:
                    break
            else:
                return
    if len(t.shape) != len(shape) or any(w is not None and int(a) != int(w)
                                         for a, w in zip(t.shape, shape)):
        want = tuple("*" if w is None else int(w) for w in shape)
        raise ValueError(f"{fn}: {name} must have shape {want}, got {tuple(t.shape)}")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{fn}: {name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous")


def _same_dtype(fn: str, **named):
    dts = {n: t.dtype for n, t in named.items() if t is not None}
    if len(set(dts.values())) > 1:
        raise ValueError(f"{fn}: {', '.join(dts)} must share one dtype, got {dts}")


def _one_device(fn: str, **named) -> torch.device:
    """Every tensor handed to the library must live on the same GPU: a host pointer reaching a
    kernel would fault the device."""
    dev = None
    for name, t in named.items():
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{fn}: {name} must be a GPU tensor, got one on {t.device}")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{fn}: {name} is on {t.device}, the other tensors on {dev}")
    return dev


def _torch_stream(stream, device):
    """The torch stream the work goes to: None = the current stream of `device`; a raw
    hipStream_t (int) is wrapped.  Outputs and workspaces the binding allocates are allocated on
    this stream, so the caching allocator never hands their memory to other work while the
    library's kernels may still use it."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream, device=device)
    return stream


def _sptr(ts) -> ctypes.c_void_p:
    return ctypes.c_void_p(ts.cuda_stream)


def _check(fn: str, status: int):
    if status != KDA_OK:
        raise KDAError(fn, status)


def kda_status_string(status: int) -> str:
    return load_library().kda_status_string(int(status)).decode()


def kda_version() -> int:
    return int(load_library().kda_version())


def kda_gate(A: torch.Tensor, z: torch.Tensor, g: Optional[torch.Tensor] = None,
             g_dtype: torch.dtype = torch.float32, g_min: float = -5.0, stream=None) -> torch.Tensor:
    """g = g_min * sigmoid(exp(A) * z); A [H, dk] fp32, z [..., H, dk] -> g like z (g_dtype)."""
    fn = "kda_gate"
    _expect(fn, "A", A, (None, None), (torch.float32,))
    H, dk = A.shape
    if z.dim() < 2:
        raise ValueError(f"{fn}: z must end in [H, dk]")
    _expect(fn, "z", z, tuple(z.shape[:-2]) + (H, dk), _FLOATS)
    _expect(fn, "g", g, tuple(z.shape), _FLOATS)
    dev = _one_device(fn, A=A, z=z, g=g)
    ts = _torch_stream(stream, dev)
    if g is None:
        with torch.cuda.stream(ts):
            g = torch.empty(z.shape, dtype=g_dtype, device=dev)
    n_tokens = z.numel() // (H * dk)
    _check(fn, load_library().kda_gate(_ptr(A), _ptr(z), _dt(z), _ptr(g), _dt(g), n_tokens, H,
                                       dk, float(g_min), _sptr(ts)))
    return g


def kda_chunk_fwd_workspace_size(n_seqs: int, total_tokens: int, H: int, dk: int, dv: int,
                                 chunk: int = 64, in_dtype: torch.dtype = torch.bfloat16) -> int:
    return int(load_library().kda_chunk_fwd_workspace_size(n_seqs, total_tokens, H, dk, dv,
                                                            chunk, _DT[in_dtype]))


def _check_prefill(fn, q, k, v, beta, gz, initial_state, final_state, cu_seqlens, o, workspace,
                   A=None, checkpoints=None):
    """Shapes, dtypes and devices of a prefill call, checked on the host before the library is
    called.  Returns (B, T, N, H, dk, dv, device)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError(f"{fn}: q must be a [B, T, H, dk] tensor")
    B, T, H, dk = (int(x) for x in q.shape)
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError(f"{fn}: v must be a [B, T, H, dv] tensor")
    dv = int(v.shape[-1])
    _expect(fn, "q", q, (B, T, H, dk), _FLOATS)
    _expect(fn, "k", k, (B, T, H, dk), _FLOATS)
    _expect(fn, "v", v, (B, T, H, dv), _FLOATS)
    _expect(fn, "beta", beta, (B, T, H), _FLOATS)
    _same_dtype(fn, q=q, k=k, v=v, beta=beta)
    _expect(fn, "g" if A is None else "z", gz, (B, T, H, dk), _FLOATS)
    _expect(fn, "A", A, (H, dk), (torch.float32,))
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError(f"{fn}: cu_seqlens needs B == 1 (a packed batch)")
        _expect(fn, "cu_seqlens", cu_seqlens, (None,), (torch.int32,))
        if cu_seqlens.numel() < 2:
            raise ValueError(f"{fn}: cu_seqlens needs at least two offsets")
    N = B if cu_seqlens is None else int(cu_seqlens.numel()) - 1
    _expect(fn, "initial_state", initial_state, (N, H, dk, dv), (torch.float32,))
    _expect(fn, "final_state", final_state, (N, H, dk, dv), (torch.float32,))
    _expect(fn, "o", o, (B, T, H, dv), _FLOATS)
    _expect(fn, "checkpoints", checkpoints, (None, H, dk, dv), (torch.float32,))
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be contiguous")
    dev = _one_device(fn, q=q, k=k, v=v, beta=beta, gz=gz, A=A, initial_state=initial_state,
                      final_state=final_state, cu_seqlens=cu_seqlens, o=o, workspace=workspace,
                      checkpoints=checkpoints)
    return B, T, N, H, dk, dv, dev


def _chunk_outputs(q, B, T, N, H, dk, dv, o, o_dtype, final_state, output_final_state,
                   workspace, ts):
    """Allocate (on the launch stream) what the caller did not pass."""
    with torch.cuda.stream(ts):
        if o is None:
            o = torch.empty((B, T, H, dv), dtype=o_dtype or q.dtype, device=q.device)
        if final_state is None and output_final_state:
            final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
        need = kda_chunk_fwd_workspace_size(N, B * T, H, dk, dv, in_dtype=q.dtype)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return o, final_state, workspace, ws_bytes


def kda_chunk_fwd(q, k, v, beta, g, initial_state=None, final_state=None, cu_seqlens=None,
                  o=None, o_dtype=None, scale: float = 1.0, output_final_state: bool = True,
                  workspace=None, stream=None):
    """Chunked prefill.  q, k, g [B, T, H, dk]; v [B, T, H, dv]; beta [B, T, H];
    initial_state [N, H, dk, dv] fp32 or None; cu_seqlens device int32 [N+1] or None (B == 1).
    Returns (o, final_state); final_state is allocated when output_final_state and not given."""
    fn = "kda_chunk_fwd"
    B, T, N, H, dk, dv, dev = _check_prefill(fn, q, k, v, beta, g, initial_state, final_state,
                                             cu_seqlens, o, workspace)
    ts = _torch_stream(stream, dev)
    o, final_state, workspace, ws_bytes = _chunk_outputs(
        q, B, T, N, H, dk, dv, o, o_dtype, final_state, output_final_state, workspace, ts)
    _check(fn, load_library().kda_chunk_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _dt(q), _ptr(g), _dt(g), _ptr(initial_state),
        _ptr(final_state), _ptr(cu_seqlens), _ptr(o), _dt(o), B, T, N, H, dk, dv, 64,
        float(scale), _ptr(workspace), ws_bytes, _sptr(ts)))
    return o, final_state


def kda_chunk_fwd_gated(q, k, v, beta, A, z, g_min: float = -5.0, initial_state=None,
                        final_state=None, cu_seqlens=None, o=None, o_dtype=None,
                        scale: float = 1.0, output_final_state: bool = True, workspace=None,
                        stream=None):
    """Chunked prefill with the gate fused: A [H, dk] fp32 and z [B, T, H, dk] replace g.
    Same outputs as kda_gate followed by kda_chunk_fwd (fp32 g)."""
    fn = "kda_chunk_fwd_gated"
    B, T, N, H, dk, dv, dev = _check_prefill(fn, q, k, v, beta, z, initial_state, final_state,
                                             cu_seqlens, o, workspace, A=A)
    ts = _torch_stream(stream, dev)
    o, final_state, workspace, ws_bytes = _chunk_outputs(
        q, B, T, N, H, dk, dv, o, o_dtype, final_state, output_final_state, workspace, ts)
    _check(fn, load_library().kda_chunk_fwd_gated(
        _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _dt(q), _ptr(A), _ptr(z), _dt(z), float(g_min),
        _ptr(initial_state), _ptr(final_state), _ptr(cu_seqlens), _ptr(o), _dt(o), B, T, N, H,
        dk, dv, 64, float(scale), _ptr(workspace), ws_bytes, _sptr(ts)))
    return o, final_state


def kda_chunk_fwd_gated_noalloc(q, k, v, beta, A, z, o, final_state=None, g_min: float = -5.0,
                                initial_state=None, cu_seqlens=None, scale: float = 1.0,
                                stream=None):
    """kda_chunk_fwd_gated with the workspace taken from the library's static device array
    (NOALLOC_SCRATCH_BYTES per GPU): nothing is allocated, here or in the library, so o (and
    final_state, if wanted) must be passed in.  Calls that overlap on one GPU race on the array.
    Returns (o, final_state)."""
    fn = "kda_chunk_fwd_gated_noalloc"
    if o is None:
        raise ValueError(f"{fn}: o must be given (nothing is allocated)")
    B, T, N, H, dk, dv, dev = _check_prefill(fn, q, k, v, beta, z, initial_state, final_state,
                                             cu_seqlens, o, None, A=A)
    ts = _torch_stream(stream, dev)
    _check(fn, load_library().kda_chunk_fwd_gated_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _dt(q), _ptr(A), _ptr(z), _dt(z), float(g_min),
        _ptr(initial_state), _ptr(final_state), _ptr(cu_seqlens), _ptr(o), _dt(o), B, T, N, H,
        dk, dv, 64, float(scale), _sptr(ts)))
    return o, final_state


def checkpoint_layout(every: int, T: int, B: int = 1, seqlens=None):
    """Host-side slot layout of kda_chunk_fwd_checkpointed: ([(first slot, count) per sequence],
    slots needed).  seqlens (host ints) describe a packed batch of total length T, else B
    sequences of T tokens."""
    if seqlens is None:
        per = T // every
        return [(n * per, per) for n in range(B)], B * per
    out, start = [], 0
    for n, length in enumerate(seqlens):
        out.append((start // every + n, int(length) // every))
        start += int(length)
    return out, T // every + len(seqlens)


def kda_chunk_fwd_checkpointed(q, k, v, beta, every: int, g=None, A=None, z=None,
                               g_min: float = -5.0, initial_state=None, final_state=None,
                               cu_seqlens=None, o=None, o_dtype=None, scale: float = 1.0,
                               output_final_state: bool = True, checkpoints=None, workspace=None,
                               stream=None):
    """Chunked prefill that also stores the state after every `every` tokens (a multiple of
    64) of each sequence.  Give g (as kda_chunk_fwd) or A and z (as kda_chunk_fwd_gated).
    Returns (o, final_state, checkpoints [slots, H, dk, dv] fp32); slot layout as
    checkpoint_layout; a new checkpoints buffer starts zeroed."""
    fn = "kda_chunk_fwd_checkpointed"
    if (g is None) == (A is None or z is None):
        raise ValueError("give either g, or A and z")
    gz = g if g is not None else z
    B, T, N, H, dk, dv, dev = _check_prefill(fn, q, k, v, beta, gz, initial_state, final_state,
                                             cu_seqlens, o, workspace, A=A,
                                             checkpoints=checkpoints)
    ts = _torch_stream(stream, dev)
    o, final_state, workspace, ws_bytes = _chunk_outputs(
        q, B, T, N, H, dk, dv, o, o_dtype, final_state, output_final_state, workspace, ts)
    need = (B * (T // every)) if cu_seqlens is None else (T // every + N)
    if checkpoints is None:
        with torch.cuda.stream(ts):
            checkpoints = torch.zeros((need, H, dk, dv), dtype=torch.float32, device=dev)
    _check(fn, load_library().kda_chunk_fwd_checkpointed(
        _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _dt(q), _ptr(A), _ptr(gz), _dt(gz), float(g_min),
        _ptr(initial_state), _ptr(final_state), _ptr(cu_seqlens), _ptr(o), _dt(o), B, T, N, H,
        dk, dv, 64, float(scale), _ptr(checkpoints), int(every), checkpoints.shape[0],
        _ptr(workspace), ws_bytes, _sptr(ts)))
    return o, final_state, checkpoints


def _check_decode(fn, q, k, v, beta, g, state, o, draft: bool, accepted=None):
    """Shapes, dtypes and devices of the decode calls: [N, H, d] per token, or [N, K, H, d]
    for a draft of K tokens.  Returns (N, K, H, dk, dv, device)."""
    nd = 4 if draft else 3
    if not isinstance(q, torch.Tensor) or q.dim() != nd:
        raise ValueError(f"{fn}: q must be a {'[N, K, H, dk]' if draft else '[N, H, dk]'} tensor")
    if not isinstance(v, torch.Tensor) or v.dim() != nd:
        raise ValueError(f"{fn}: v must have {nd} dimensions")
    lead = tuple(int(x) for x in q.shape[:-1])
    N, H, dk, dv = lead[0], lead[-1], int(q.shape[-1]), int(v.shape[-1])
    K = lead[1] if draft else 1
    _expect(fn, "q", q, lead + (dk,), _FLOATS)
    _expect(fn, "k", k, lead + (dk,), _FLOATS)
    _expect(fn, "v", v, lead + (dv,), _FLOATS)
    _expect(fn, "beta", beta, lead, _FLOATS)
    _same_dtype(fn, q=q, k=k, v=v, beta=beta)
    _expect(fn, "g", g, lead + (dk,), _FLOATS)
    _expect(fn, "state", state, (N, H, dk, dv), (torch.float32,))
    _expect(fn, "o", o, lead + (dv,), _FLOATS)
    _expect(fn, "accepted", accepted, (N,), (torch.int32,))
    dev = _one_device(fn, q=q, k=k, v=v, beta=beta, g=g, state=state, o=o, accepted=accepted)
    return N, K, H, dk, dv, dev


def kda_decode_step(q, k, v, beta, g, state, o=None, o_dtype=None, scale: float = 1.0,
                    stream=None):
    """One token per sequence: q, k, g [N, H, dk]; v [N, H, dv]; beta [N, H]; state
    [N, H, dk, dv] fp32 updated in place.  Returns o [N, H, dv]."""
    fn = "kda_decode_step"
    N, _, H, dk, dv, dev = _check_decode(fn, q, k, v, beta, g, state, o, draft=False)
    ts = _torch_stream(stream, dev)
    if o is None:
        with torch.cuda.stream(ts):
            o = torch.empty((N, H, dv), dtype=o_dtype or q.dtype, device=dev)
    _check(fn, load_library().kda_decode_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _dt(q), _ptr(g), _dt(g), _ptr(state), _ptr(o),
        _dt(o), N, H, dk, dv, float(scale), _sptr(ts)))
    return o


def kda_decode_verify(q, k, v, beta, g, state, o=None, o_dtype=None, scale: float = 1.0,
                      stream=None):
    """K draft tokens per sequence from a read-only state: q, k, g [N, K, H, dk]; v [N, K, H, dv];
    beta [N, K, H]; state [N, H, dk, dv] fp32 (not modified).  Returns o [N, K, H, dv]."""
    fn = "kda_decode_verify"
    N, Kd, H, dk, dv, dev = _check_decode(fn, q, k, v, beta, g, state, o, draft=True)
    ts = _torch_stream(stream, dev)
    if o is None:
        with torch.cuda.stream(ts):
            o = torch.empty((N, Kd, H, dv), dtype=o_dtype or q.dtype, device=dev)
    _check(fn, load_library().kda_decode_verify(
        _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _dt(q), _ptr(g), _dt(g), _ptr(state), _ptr(o),
        _dt(o), N, Kd, H, dk, dv, float(scale), _sptr(ts)))
    return o


def kda_decode_commit(q, k, v, beta, g, state, accepted, stream=None):
    """Advance each state in place by its first accepted[n] draft tokens (device int32 [N]);
    inputs as kda_decode_verify.  Returns state."""
    fn = "kda_decode_commit"
    if not isinstance(accepted, torch.Tensor) or accepted.dtype != torch.int32:
        raise TypeError(f"{fn}: accepted must be an int32 tensor")
    N, Kd, H, dk, dv, dev = _check_decode(fn, q, k, v, beta, g, state, None, draft=True,
                                          accepted=accepted)
    ts = _torch_stream(stream, dev)
    _check(fn, load_library().kda_decode_commit(
        _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _dt(q), _ptr(g), _dt(g), _ptr(state),
        _ptr(accepted), N, Kd, H, dk, dv, _sptr(ts)))
    return state


# ---- linear attention with one decay per head ---------------------------------------------------

def _launch_stream(stream, dev):
    """(torch stream or None for the current one of `dev`, its raw pointer)."""
    if stream is None:
        return None, torch._C._cuda_getCurrentRawStream(dev.index)
    ts = _torch_stream(stream, dev)
    return ts, ts.cuda_stream


def _launch(fn: str, dev: torch.device, call, *args):
    """call(*args) with `dev` current; raises for a status other than KDA_OK."""
    if torch._C._cuda_getDevice() == dev.index:
        status = call(*args)
    else:
        with torch.cuda.device(dev):
            status = call(*args)
    if status != KDA_OK:
        raise KDAError(fn, status)


def _fit(dev, *specs) -> bool:
    """Whether every (tensor or None, shape, dtype) of `specs` is as stated, contiguous and on `dev`:
    the quick form of the checks that _expect and _one_device make (and word) one by one."""
    for t, shape, dtype in specs:
        if t is not None and not (isinstance(t, torch.Tensor) and t.shape == shape and
                                  t.dtype is dtype and t.device == dev and t.is_contiguous()):
            return False
    return dev.type == "cuda"


def _size(t, dims: int, d: int):
    """Size d of a tensor of `dims` dimensions, None for anything else."""
    return t.shape[d] if isinstance(t, torch.Tensor) and t.dim() == dims else None


def _alloc(ts, shape, dtype, dev):
    """A new tensor on the launch stream `ts` (None: the current one)."""
    if ts is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(ts):
        return torch.empty(shape, dtype=dtype, device=dev)


def _addr(t: Optional[torch.Tensor]):
    """Address of a tensor that has passed _expect."""
    return None if t is None else t.data_ptr()


def kda_linear_chunk_workspace_size(n_seqs: int, total_tokens: int, H: int, dk: int, dv: int,
                                    in_dtype: torch.dtype = torch.bfloat16,
                                    backward: bool = False) -> int:
    return int(load_library().kda_linear_chunk_workspace_size(n_seqs, total_tokens, H, dk, dv,
                                                              _DT[in_dtype], int(backward)))


def _check_linear(fn, q, k, v, g, cu_seqlens, workspace, states, like_q, like_v):
    """Shapes, dtypes and devices of a linear-attention prefill or backward call.  `states`,
    `like_q` and `like_v` map argument names to tensors shaped as a state, q or v.  Returns
    (B, T, N, H, dk, dv, device)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError(f"{fn}: q must be a [B, T, H, dk] tensor")
    B, T, H, dk = q.shape
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError(f"{fn}: v must be a [B, T, H, dv] tensor")
    dv = v.shape[-1]
    _expect(fn, "q", q, (B, T, H, dk), _FLOATS)
    _expect(fn, "k", k, (B, T, H, dk), _FLOATS)
    _expect(fn, "v", v, (B, T, H, dv), _FLOATS)
    _same_dtype(fn, q=q, k=k, v=v)
    _expect(fn, "g", g, (H,), (torch.float32,))
    N = B
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError(f"{fn}: cu_seqlens needs B == 1 (a packed batch)")
        _expect(fn, "cu_seqlens", cu_seqlens, (None,), (torch.int32,))
        N = cu_seqlens.numel() - 1
        if N < 1:
            raise ValueError(f"{fn}: cu_seqlens needs at least two offsets")
    for name, t in states.items():
        _expect(fn, name, t, (N, H, dk, dv), (torch.float32,))
    for name, t in like_q.items():
        _expect(fn, name, t, (B, T, H, dk), (q.dtype,))
    for name, t in like_v.items():
        _expect(fn, name, t, (B, T, H, dv), _FLOATS if name == "o" else (q.dtype,))
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be contiguous")
    dev = _one_device(fn, q=q, k=k, v=v, g=g, cu_seqlens=cu_seqlens, workspace=workspace, **states,
                      **like_q, **like_v)
    return B, T, N, H, dk, dv, dev


def _linear_workspace(ts, workspace, N, ntok, H, dk, dv, dtype, backward, dev):
    """The workspace (allocated on `ts` where none is given and one is needed) and its bytes."""
    if workspace is None:
        need = kda_linear_chunk_workspace_size(N, ntok, H, dk, dv, dtype, backward)
        if need == 0:
            return None, 0
        workspace = _alloc(ts, (need,), torch.uint8, dev)
    return workspace, workspace.numel() * workspace.element_size()


def kda_linear_chunk_fwd(q, k, v, g, initial_state=None, final_state=None, cu_seqlens=None, o=None,
                         o_dtype=None, scale: float = 1.0, output_final_state: bool = True,
                         workspace=None, stream=None):
    """Chunked prefill of linear attention, S_t = e^g S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t:
    q, k [B, T, H, dk]; v [B, T, H, dv]; g [H] fp32 log-decay (<= 0); initial_state
    [N, H, dk, dv] fp32 or None; cu_seqlens device int32 [N+1] or None (B == 1).  Returns
    (o, final_state); final_state is allocated when output_final_state and not given.  Not recorded by
    autograd: gradients come from kda_linear_chunk_bwd."""
    fn = "kda_linear_chunk_fwd"
    B, T, N, H, dk, dv, dev = _check_linear(
        fn, q, k, v, g, cu_seqlens, workspace,
        dict(initial_state=initial_state, final_state=final_state), {}, dict(o=o))
    ts, sp = _launch_stream(stream, dev)
    if o is None:
        o = _alloc(ts, (B, T, H, dv), o_dtype or q.dtype, dev)
    if final_state is None and output_final_state:
        final_state = _alloc(ts, (N, H, dk, dv), torch.float32, dev)
    workspace, ws_bytes = _linear_workspace(ts, workspace, N, B * T, H, dk, dv, q.dtype, False, dev)
    _launch(fn, dev, load_library().kda_linear_chunk_fwd, _addr(q), _addr(k), _addr(v), _dt(q),
            _addr(g), _addr(initial_state), _addr(final_state), _addr(cu_seqlens), _addr(o), _dt(o),
            B, T, N, H, dk, dv, float(scale), _addr(workspace), ws_bytes, sp)
    return o, final_state


def kda_linear_chunk_bwd(q, k, v, g, do, initial_state=None, d_final_state=None, cu_seqlens=None,
                         dq=None, dk=None, dv=None, d_initial_state=None, scale: float = 1.0,
                         output_d_initial_state: Optional[bool] = None, workspace=None,
                         stream=None):
    """Gradients of kda_linear_chunk_fwd: do [B, T, H, dv] in q's dtype, d_final_state
    [N, H, dk, dv] fp32 or None (zeros), the other inputs as there.  Returns (dq, dk, dv,
    d_initial_state); the last is allocated when output_d_initial_state (default: when
    initial_state is given) and not given, else None."""
    fn = "kda_linear_chunk_bwd"
    if not isinstance(do, torch.Tensor):
        raise TypeError(f"{fn}: do must be a torch.Tensor")
    B, T, N, H, d_k, d_v, dev = _check_linear(
        fn, q, k, v, g, cu_seqlens, workspace,
        dict(initial_state=initial_state, d_final_state=d_final_state,
             d_initial_state=d_initial_state), dict(dq=dq, dk=dk), dict(do=do, dv=dv))
    ts, sp = _launch_stream(stream, dev)
    if dq is None:
        dq = _alloc(ts, q.shape, q.dtype, dev)
    if dk is None:
        dk = _alloc(ts, q.shape, q.dtype, dev)
    if dv is None:
        dv = _alloc(ts, v.shape, q.dtype, dev)
    if output_d_initial_state is None:
        output_d_initial_state = initial_state is not None
    if d_initial_state is None and output_d_initial_state:
        d_initial_state = _alloc(ts, (N, H, d_k, d_v), torch.float32, dev)
    workspace, ws_bytes = _linear_workspace(ts, workspace, N, B * T, H, d_k, d_v, q.dtype, True, dev)
    _launch(fn, dev, load_library().kda_linear_chunk_bwd, _addr(q), _addr(k), _addr(v), _dt(q),
            _addr(g), _addr(initial_state), _addr(cu_seqlens), _addr(do), _addr(d_final_state),
            _addr(dq), _addr(dk), _addr(dv), _addr(d_initial_state), B, T, N, H, d_k, d_v,
            float(scale), _addr(workspace), ws_bytes, sp)
    return dq, dk, dv, d_initial_state


def kda_linear_decode_step(q, k, v, g, state, o=None, o_dtype=None, scale: float = 1.0,
                           stream=None):
    """One token of linear attention per sequence: q, k [N, H, dk]; v [N, H, dv]; g [H] fp32;
    state [N, H, dk, dv] fp32 updated in place.  Returns o [N, H, dv]."""
    fn = "kda_linear_decode_step"
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError(f"{fn}: q must be a [N, H, dk] tensor")
    if not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError(f"{fn}: v must be a [N, H, dv] tensor")
    N, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    if o is not None or dt not in _FLOATS or not _fit(
            dev, (q, (N, H, dk), dt), (k, (N, H, dk), dt), (v, (N, H, dv), dt), (g, (H,), torch.float32),
            (state, (N, H, dk, dv), torch.float32)):
        _expect(fn, "q", q, (N, H, dk), _FLOATS)
        _expect(fn, "k", k, (N, H, dk), _FLOATS)
        _expect(fn, "v", v, (N, H, dv), _FLOATS)
        _same_dtype(fn, q=q, k=k, v=v)
        _expect(fn, "g", g, (H,), (torch.float32,))
        _expect(fn, "state", state, (N, H, dk, dv), (torch.float32,))
        _expect(fn, "o", o, (N, H, dv), _FLOATS)
        _one_device(fn, q=q, k=k, v=v, g=g, state=state, o=o)
    ts, sp = _launch_stream(stream, dev)
    if o is None:
        o = _alloc(ts, (N, H, dv), o_dtype or q.dtype, dev)
    _launch(fn, dev, load_library().kda_linear_decode_step, _addr(q), _addr(k), _addr(v), _dt(q),
            _addr(g), _addr(state), _addr(o), _dt(o), N, H, dk, dv, float(scale), sp)
    return o


# ---- 8-bit state cache --------------------------------------------------------------------------

KDA_CODE_I8, KDA_CODE_E4M3 = 0, 1
_CODES = {torch.int8: KDA_CODE_I8, torch.float8_e4m3fn: KDA_CODE_E4M3}


def _check_cache(fn, codes, scales, slots, states):
    """Shapes, dtypes and devices of a state-cache call; states may be None (to be allocated).
    Returns (N, n_slots, H, dk, dv, group, device)."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 4:
        raise ValueError(f"{fn}: codes must be a [n_slots, H, dk, dv] tensor")
    n_slots, H, dk, dv = codes.shape
    dev = codes.device
    groups = scales.shape[-1] if isinstance(scales, torch.Tensor) and scales.dim() == 4 else 0
    if slots is not None and codes.dtype in _CODES and groups > 0 and dv % groups == 0 and \
            isinstance(slots, torch.Tensor) and slots.dim() == 1:
        N = slots.shape[0]
        if _fit(dev, (codes, (n_slots, H, dk, dv), codes.dtype), (slots, (N,), torch.int32),
                (scales, (n_slots, H, dk, groups), torch.float32), (states, (N, H, dk, dv), torch.float32)):
            return N, n_slots, H, dk, dv, dv // groups, dev
    _expect(fn, "codes", codes, (n_slots, H, dk, dv), tuple(_CODES))
    if not isinstance(scales, torch.Tensor):
        raise TypeError(f"{fn}: scales must be a torch.Tensor")
    _expect(fn, "scales", scales, (n_slots, H, dk, None), (torch.float32,))
    if scales.shape[-1] < 1 or dv % scales.shape[-1] != 0:
        raise ValueError(f"{fn}: scales must end in dv / group, got {scales.shape[-1]} for dv = {dv}")
    _expect(fn, "slots", slots, (None,), (torch.int32,))
    N = slots.numel() if slots is not None else (n_slots if states is None else states.shape[0])
    _expect(fn, "states", states, (N, H, dk, dv), (torch.float32,))
    dev = _one_device(fn, codes=codes, scales=scales, slots=slots, states=states)
    return N, n_slots, H, dk, dv, dv // scales.shape[-1], dev


def kda_state_store(states, codes, scales, slots=None, stream=None):
    """Writes states [N, H, dk, dv] fp32 into slots slots[n] (device int32 [N]; None: slot n) of the
    8-bit state cache: codes [n_slots, H, dk, dv] (torch.int8 or torch.float8_e4m3fn) and scales
    [n_slots, H, dk, dv / group] fp32, group 32, 64 or 128.  Slots outside the cache are skipped; of
    several states for one slot the last is stored.  Returns (codes, scales)."""
    fn = "kda_state_store"
    if not isinstance(states, torch.Tensor) or states.dim() != 4:
        raise ValueError(f"{fn}: states must be a [N, H, dk, dv] tensor")
    N, n_slots, H, dk, dv, group, dev = _check_cache(fn, codes, scales, slots, states)
    _, sp = _launch_stream(stream, dev)
    _launch(fn, dev, load_library().kda_state_store, _addr(states), _addr(slots), _addr(codes),
            _CODES[codes.dtype], _addr(scales), N, n_slots, H, dk, dv, group, sp)
    return codes, scales


def kda_state_load(codes, scales, slots=None, states=None, stream=None):
    """Reads states back: states[n] = codes * scales of slot slots[n] (None: slot n), zeros where the
    slot lies outside the cache (-1: no cached prefix).  Returns states [N, H, dk, dv] fp32."""
    fn = "kda_state_load"
    N, n_slots, H, dk, dv, group, dev = _check_cache(fn, codes, scales, slots, states)
    ts, sp = _launch_stream(stream, dev)
    if states is None:
        states = _alloc(ts, (N, H, dk, dv), torch.float32, dev)
    _launch(fn, dev, load_library().kda_state_load, _addr(codes), _CODES[codes.dtype],
            _addr(scales), _addr(slots), _addr(states), N, n_slots, H, dk, dv, group, sp)
    return states


# ---- rows of tokens that may be parts of wider rows ---------------------------------------------

def _rows(fn, name, t, shape, dtype, lead):
    """Elements from one token's row of t to the next: t has the given shape, its first `lead`
    dimensions count tokens, the others are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{fn}: {name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{fn}: {name} must be {dtype}, got {t.dtype}")
    row = 1
    for n in shape[lead:]:
        row *= n
    if t.is_contiguous():
        return row
    strides, want = t.stride(), 1
    for d in range(len(shape) - 1, lead - 1, -1):
        if shape[d] != 1 and strides[d] != want:
            raise ValueError(f"{fn}: {name}'s rows must be contiguous")
        want *= shape[d]
    ld, tokens = None, 1
    for d in range(lead - 1, -1, -1):
        if shape[d] != 1:
            if ld is None:
                ld = strides[d]
            elif strides[d] != ld * tokens:
                raise ValueError(f"{fn}: {name}'s tokens must be evenly spaced")
        tokens *= shape[d]
    if ld is None or tokens == 0:
        return row
    if ld < row:
        raise ValueError(f"{fn}: {name}'s rows must not overlap")
    return ld


def _required(fn, **named):
    """Tensors that the call cannot do without (_expect takes None for an absent one)."""
    for name, t in named.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{fn}: {name} must be a torch.Tensor")


def _float_dtype(fn, name, t):
    if not isinstance(t, torch.Tensor) or t.dtype not in _FLOATS:
        raise TypeError(f"{fn}: {name} must be a float32 or bfloat16 tensor")
    return t.dtype


def _sequences(fn, B, cu_seqlens):
    """Sequences of a batch of B rows of tokens, or of a packed one."""
    if cu_seqlens is None:
        return B
    if B != 1:
        raise ValueError(f"{fn}: cu_seqlens needs B == 1 (a packed batch)")
    _expect(fn, "cu_seqlens", cu_seqlens, (None,), (torch.int32,))
    if cu_seqlens.numel() < 2:
        raise ValueError(f"{fn}: cu_seqlens needs at least two offsets")
    return cu_seqlens.numel() - 1


def _bytes_of(fn, ts, workspace, need, dev):
    """The workspace (allocated on `ts` where none is given and one is needed) and its bytes."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = _alloc(ts, (need,), torch.uint8, dev)
    elif not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


# ---- short convolution --------------------------------------------------------------------------

def _check_conv(fn, x, weight, bias, cu_seqlens, like_x, windows):
    """Sizes and strides of a convolution's prompt calls: (B, T, N, C, W, ldx, strides of like_x)."""
    dt = _float_dtype(fn, "x", x)
    if x.dim() != 3:
        raise ValueError(f"{fn}: x must be a [B, T, C] tensor")
    B, T, C = x.shape
    ldx = _rows(fn, "x", x, (B, T, C), dt, 2)
    _required(fn, weight=weight)
    _expect(fn, "weight", weight, (C, None), (torch.float32,))
    _expect(fn, "bias", bias, (C,), (torch.float32,))
    W = weight.shape[1]
    N = _sequences(fn, B, cu_seqlens)
    lds = [ldx if t is None else _rows(fn, name, t, (B, T, C), dt, 2) for name, t in like_x.items()]
    for name, t in windows.items():
        _expect(fn, name, t, (N, W - 1, C), (dt,))
    return B, T, N, C, W, ldx, lds


def kda_conv_fwd(x, weight, bias=None, initial_state=None, final_state=None, cu_seqlens=None, y=None,
                 silu: bool = True, output_final_state: bool = False, stream=None):
    """Short causal convolution of every channel, u_t = bias + sum_i weight[:, i] x_{t-W+1+i} and
    y = silu(u) (or u): x [B, T, C], whose rows may be parts of wider ones; weight [C, W] fp32 with W
    2, 3 or 4; bias [C] fp32 or None; initial_state [N, W-1, C] in x's dtype or None (zeros); cu_seqlens
    device int32 [N+1] or None (B == 1).  Returns (y, final_state), the latter the last W - 1
    inputs, allocated when output_final_state and not given.  Not recorded by autograd: gradients come
    from kda_conv_bwd."""
    fn = "kda_conv_fwd"
    B, T, N, C, W, ldx, (ldy,) = _check_conv(
        fn, x, weight, bias, cu_seqlens, dict(y=y),
        dict(initial_state=initial_state, final_state=final_state))
    dev = _one_device(fn, x=x, weight=weight, bias=bias, initial_state=initial_state,
                      final_state=final_state, cu_seqlens=cu_seqlens, y=y)
    ts, sp = _launch_stream(stream, dev)
    if y is None:
        y, ldy = _alloc(ts, (B, T, C), x.dtype, dev), C
    if final_state is None and output_final_state:
        final_state = _alloc(ts, (N, W - 1, C), x.dtype, dev)
    _launch(fn, dev, load_library().kda_conv_fwd, _addr(x), ldx, _dt(x), _addr(weight), _addr(bias),
            _addr(initial_state), _addr(final_state), _addr(cu_seqlens), _addr(y), ldy, B, T, N, C, W,
            int(silu), sp)
    return y, final_state


def kda_conv_bwd_workspace_size(n_seqs: int, total_tokens: int, C: int, W: int) -> int:
    return int(load_library().kda_conv_bwd_workspace_size(n_seqs, total_tokens, C, W))


def kda_conv_bwd(x, weight, dy, bias=None, initial_state=None, d_final_state=None, cu_seqlens=None,
                 silu: bool = True, dx=None, output_d_initial_state: Optional[bool] = None,
                 workspace=None, stream=None):
    """Gradients of kda_conv_fwd: dy [B, T, C] and d_final_state [N, W-1, C] (or None: zeros) in x's
    dtype, the other inputs as there.  Returns (dx, d_weight, d_bias, d_initial_state); d_bias is
    None without a bias, d_initial_state is formed when output_d_initial_state (default: when
    initial_state is given)."""
    fn = "kda_conv_bwd"
    if not isinstance(dy, torch.Tensor):
        raise TypeError(f"{fn}: dy must be a torch.Tensor")
    B, T, N, C, W, ldx, (lddy, lddx) = _check_conv(
        fn, x, weight, bias, cu_seqlens, dict(dy=dy, dx=dx),
        dict(initial_state=initial_state, d_final_state=d_final_state))
    dev = _one_device(fn, x=x, weight=weight, dy=dy, bias=bias, initial_state=initial_state,
                      d_final_state=d_final_state, cu_seqlens=cu_seqlens, dx=dx, workspace=workspace)
    ts, sp = _launch_stream(stream, dev)
    if dx is None:
        dx, lddx = _alloc(ts, (B, T, C), x.dtype, dev), C
    d_weight = _alloc(ts, (C, W), torch.float32, dev)
    d_bias = None if bias is None else _alloc(ts, (C,), torch.float32, dev)
    if output_d_initial_state is None:
        output_d_initial_state = initial_state is not None
    dh0 = _alloc(ts, (N, W - 1, C), x.dtype, dev) if output_d_initial_state else None
    workspace, ws_bytes = _bytes_of(fn, ts, workspace, kda_conv_bwd_workspace_size(N, B * T, C, W), dev)
    _launch(fn, dev, load_library().kda_conv_bwd, _addr(x), ldx, _dt(x), _addr(weight), _addr(bias),
            _addr(initial_state), _addr(cu_seqlens), _addr(dy), lddy, _addr(d_final_state), _addr(dx), lddx,
            _addr(d_weight), _addr(d_bias), _addr(dh0), B, T, N, C, W, int(silu), _addr(workspace),
            ws_bytes, sp)
    return dx, d_weight, d_bias, dh0


def kda_conv_step(x, weight, windows, bias=None, slots=None, y=None, silu: bool = True, stream=None):
    """One token of kda_conv_fwd for N sequences: x [N, C]; windows [n_slots, W-1, C] in x's dtype, moved
    on in place; slots device int32 [N] or None (sequence n in slot n).  Sequences whose slot lies
    outside the pool, and all but the last with one slot, are skipped and get zeros.  Returns y [N, C]."""
    fn = "kda_conv_step"
    dt = _float_dtype(fn, "x", x)
    if x.dim() != 2:
        raise ValueError(f"{fn}: x must be a [N, C] tensor")
    N, C = x.shape
    dev, W, n_slots = x.device, _size(weight, 2, 1), _size(windows, 3, 0)
    ldx = ldy = C
    if y is not None or not W or n_slots is None or not _fit(
            dev, (x, (N, C), dt), (weight, (C, W), torch.float32), (windows, (n_slots, W - 1, C), dt),
            (bias, (C,), torch.float32), (slots, (N,), torch.int32)):
        ldx = _rows(fn, "x", x, (N, C), dt, 1)
        _required(fn, weight=weight, windows=windows)
        _expect(fn, "weight", weight, (C, None), (torch.float32,))
        _expect(fn, "windows", windows, (None, W - 1, C), (dt,))
        _expect(fn, "bias", bias, (C,), (torch.float32,))
        _expect(fn, "slots", slots, (N,), (torch.int32,))
        ldy = C if y is None else _rows(fn, "y", y, (N, C), dt, 1)
        _one_device(fn, x=x, weight=weight, windows=windows, bias=bias, slots=slots, y=y)
    ts, sp = _launch_stream(stream, dev)
    if y is None:
        y = _alloc(ts, (N, C), dt, dev)
    _launch(fn, dev, load_library().kda_conv_step, _addr(x), ldx, _DT[dt], _addr(weight), _addr(bias),
            _addr(windows), _addr(slots), _addr(y), ldy, N, n_slots, C, W, int(silu), sp)
    return y


# ---- selective state space scan -----------------------------------------------------------------

def kda_ssm_chunk_workspace_size(n_seqs: int, total_tokens: int, H: int, G: int, dk: int, dv: int,
                                 in_dtype: torch.dtype = torch.bfloat16, backward: bool = False) -> int:
    """Bytes of a scan call's workspace.  Never falls as n_seqs or total_tokens grow: what serves the
    largest batch serves every smaller one of the same heads and type."""
    return int(load_library().kda_ssm_chunk_workspace_size(n_seqs, total_tokens, H, G, dk, dv,
                                                           _DT[in_dtype], int(backward)))


def _check_ssm(fn, x, dt, A, B, C, D, dt_bias, lead):
    """Sizes and strides of a scan's inputs, `lead` dimensions of tokens: (tokens' sizes, H, G, dk, dv,
    strides of x, dt, B, C)."""
    ty = _float_dtype(fn, "x", x)
    if x.dim() != lead + 2:
        raise ValueError(f"{fn}: x must be a {'[B, T, H, dv]' if lead == 2 else '[N, H, dv]'} tensor")
    if not isinstance(B, torch.Tensor) or B.dim() != lead + 2:
        raise ValueError(f"{fn}: B must be a {'[B, T, G, dk]' if lead == 2 else '[N, G, dk]'} tensor")
    tok, (H, dv), (G, dk) = tuple(x.shape[:lead]), x.shape[lead:], B.shape[lead:]
    if G < 1 or H % G != 0:
        raise ValueError(f"{fn}: G = {G} must divide H = {H}")
    lds = (_rows(fn, "x", x, tok + (H, dv), ty, lead), _rows(fn, "dt", dt, tok + (H,), ty, lead),
           _rows(fn, "B", B, tok + (G, dk), ty, lead), _rows(fn, "C", C, tok + (G, dk), ty, lead))
    _required(fn, A=A)
    _expect(fn, "A", A, (H,), (torch.float32,))
    _expect(fn, "D", D, (H,), (torch.float32,))
    _expect(fn, "dt_bias", dt_bias, (H,), (torch.float32,))
    return tok, H, G, dk, dv, lds


def kda_ssm_chunk_fwd(x, dt, A, B, C, D=None, dt_bias=None, initial_state=None, final_state=None,
                      cu_seqlens=None, y=None, y_dtype=None, output_final_state: bool = True,
                      workspace=None, stream=None):
    """Chunked prefill of the selective state space scan: with delta = softplus(dt + dt_bias),
    S_t = e^(delta_t A) S_{t-1} + delta_t B_t x_t^T and y_t = S_t^T C_t + D x_t.  x [B, T, H, dv];
    dt [B, T, H]; B, C [B, T, G, dk] (head h uses group h // (H // G)), whose rows may be parts of wider
    ones; A (<= 0), D, dt_bias [H] fp32, the latter two may be None; initial_state [N, H, dk, dv]
    fp32 or None; cu_seqlens device int32 [N+1] or None (B == 1).  Returns (y, final_state);
    final_state is allocated when output_final_state and not given.  Not recorded by autograd:
    gradients come from kda_ssm_chunk_bwd."""
    fn = "kda_ssm_chunk_fwd"
    (nb, T), H, G, dk, dv, (ldx, lddt, ldb, ldc) = _check_ssm(fn, x, dt, A, B, C, D, dt_bias, 2)
    N = _sequences(fn, nb, cu_seqlens)
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        _expect(fn, name, t, (N, H, dk, dv), (torch.float32,))
    ldy = H * dv if y is None else _rows(fn, "y", y, (nb, T, H, dv), _float_dtype(fn, "y", y), 2)
    dev = _one_device(fn, x=x, dt=dt, A=A, B=B, C=C, D=D, dt_bias=dt_bias, initial_state=initial_state,
                      final_state=final_state, cu_seqlens=cu_seqlens, y=y, workspace=workspace)
    ts, sp = _launch_stream(stream, dev)
    if y is None:
        y = _alloc(ts, (nb, T, H, dv), y_dtype or x.dtype, dev)
    if final_state is None and output_final_state:
        final_state = _alloc(ts, (N, H, dk, dv), torch.float32, dev)
    workspace, ws_bytes = _bytes_of(fn, ts, workspace, 0 if workspace is not None else
                                    kda_ssm_chunk_workspace_size(N, nb * T, H, G, dk, dv, x.dtype), dev)
    _launch(fn, dev, load_library().kda_ssm_chunk_fwd, _addr(x), ldx, _addr(dt), lddt, _addr(B), ldb,
            _addr(C), ldc, _dt(x), _addr(A), _addr(dt_bias), _addr(D), _addr(initial_state),
            _addr(final_state), _addr(cu_seqlens), _addr(y), ldy, _dt(y), nb, T, N, H, G, dk, dv,
            _addr(workspace), ws_bytes, sp)
    return y, final_state


def kda_ssm_chunk_bwd(x, dt, A, B, C, dy, D=None, dt_bias=None, initial_state=None, d_final_state=None,
                      cu_seqlens=None, dx=None, ddt=None, dB=None, dC=None, d_initial_state=None,
                      output_d_initial_state: Optional[bool] = None, workspace=None, stream=None):
    """Gradients of kda_ssm_chunk_fwd: dy [B, T, H, dv] in x's dtype, d_final_state [N, H, dk, dv] fp32
    or None (zeros), the other inputs as there; dx, ddt, dB, dC may be given (parts of wider rows, say).
    Returns (dx, ddt, dA, dB, dC, dD, d_dt_bias, d_initial_state); dD and d_dt_bias are None without
    D and dt_bias, d_initial_state is formed when output_d_initial_state (default: when initial_state
    is given) or given."""
    fn = "kda_ssm_chunk_bwd"
    (nb, T), H, G, dk, dv, (ldx, lddt, ldb, ldc) = _check_ssm(fn, x, dt, A, B, C, D, dt_bias, 2)
    N, ty = _sequences(fn, nb, cu_seqlens), x.dtype
    lddy = _rows(fn, "dy", dy, (nb, T, H, dv), ty, 2)
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state),
                    ("d_initial_state", d_initial_state)):
        _expect(fn, name, t, (N, H, dk, dv), (torch.float32,))
    dev = _one_device(fn, x=x, dt=dt, A=A, B=B, C=C, dy=dy, D=D, dt_bias=dt_bias,
                      initial_state=initial_state, d_final_state=d_final_state, cu_seqlens=cu_seqlens,
                      dx=dx, ddt=ddt, dB=dB, dC=dC, d_initial_state=d_initial_state, workspace=workspace)
    ts, sp = _launch_stream(stream, dev)
    outs = []
    for name, t, like in (("dx", dx, x), ("ddt", ddt, dt), ("dB", dB, B), ("dC", dC, C)):
        if t is None:
            t = _alloc(ts, like.shape, ty, dev)
        outs.append((t, _rows(fn, name, t, like.shape, ty, 2)))
    (dx, lddx), (ddt, ldddt), (dB, lddb), (dC, lddc) = outs
    heads = _alloc(ts, (3, H), torch.float32, dev)
    dA, dD, dbias = heads[0], None if D is None else heads[1], None if dt_bias is None else heads[2]
    if output_d_initial_state is None:
        output_d_initial_state = initial_state is not None
    if d_initial_state is None and output_d_initial_state:
        d_initial_state = _alloc(ts, (N, H, dk, dv), torch.float32, dev)
    workspace, ws_bytes = _bytes_of(fn, ts, workspace, 0 if workspace is not None else
                                    kda_ssm_chunk_workspace_size(N, nb * T, H, G, dk, dv, ty, True), dev)
    _launch(fn, dev, load_library().kda_ssm_chunk_bwd, _addr(x), ldx, _addr(dt), lddt, _addr(B), ldb,
            _addr(C), ldc, _dt(x), _addr(A), _addr(dt_bias), _addr(D), _addr(initial_state),
            _addr(cu_seqlens), _addr(dy), lddy, _addr(d_final_state), _addr(dx), lddx, _addr(ddt), ldddt,
            _addr(dB), lddb, _addr(dC), lddc, _addr(dA), _addr(dD), _addr(dbias), _addr(d_initial_state),
            nb, T, N, H, G, dk, dv, _addr(workspace), ws_bytes, sp)
    return dx, ddt, dA, dB, dC, dD, dbias, d_initial_state


def kda_ssm_decode_step(x, dt, A, B, C, state, D=None, dt_bias=None, slots=None, y=None, y_dtype=None,
                        stream=None):
    """One token of the selective scan for N sequences: x [N, H, dv]; dt [N, H]; B, C [N, G, dk]; A, D,
    dt_bias [H] fp32; state [n_slots, H, dk, dv] fp32 updated in place; slots device int32 [N] or None
    (sequence n in slot n).  Sequences whose slot lies outside the pool, and all but the last with one
    slot, are skipped and get zeros.  Returns y [N, H, dv]."""
    fn = "kda_ssm_decode_step"
    n_slots, f32 = _size(state, 4, 0), torch.float32
    quick = y is None and n_slots is not None and _size(x, 3, 0) is not None and _size(B, 3, 0) is not None
    if quick:
        (N, H, dv), (_, G, dk), ty, dev = x.shape, B.shape, x.dtype, x.device
        quick = ty in _FLOATS and A is not None and dt is not None and C is not None and G > 0 and H % G == 0 and _fit(
            dev, (x, (N, H, dv), ty), (dt, (N, H), ty), (B, (N, G, dk), ty), (C, (N, G, dk), ty), (A, (H,), f32),
            (D, (H,), f32), (dt_bias, (H,), f32), (state, (n_slots, H, dk, dv), f32), (slots, (N,), torch.int32))
        ldx, lddt, ldb, ldc, ldy = H * dv, H, G * dk, G * dk, H * dv
    if not quick:
        (N,), H, G, dk, dv, (ldx, lddt, ldb, ldc) = _check_ssm(fn, x, dt, A, B, C, D, dt_bias, 1)
        _required(fn, state=state)
        _expect(fn, "state", state, (None, H, dk, dv), (f32,))
        _expect(fn, "slots", slots, (N,), (torch.int32,))
        ldy = H * dv if y is None else _rows(fn, "y", y, (N, H, dv), _float_dtype(fn, "y", y), 1)
        dev = _one_device(fn, x=x, dt=dt, A=A, B=B, C=C, state=state, D=D, dt_bias=dt_bias, slots=slots, y=y)
    ts, sp = _launch_stream(stream, dev)
    if y is None:
        y = _alloc(ts, (N, H, dv), y_dtype or x.dtype, dev)
    _launch(fn, dev, load_library().kda_ssm_decode_step, _addr(x), ldx, _addr(dt), lddt, _addr(B), ldb,
            _addr(C), ldc, _dt(x), _addr(A), _addr(dt_bias), _addr(D), _addr(state), _addr(slots),
            _addr(y), ldy, _dt(y), N, n_slots, H, G, dk, dv, sp)
    return y


# ---- slot pools ---------------------------------------------------------------------------------

def _planes(fn, name, pool):
    """(number of slots, addresses, bytes of a slot, number of planes) of a pool: a tensor or a list of
    up to four, each with the slots as its first dimension."""
    pool = [pool] if isinstance(pool, torch.Tensor) else list(pool)
    if not 1 <= len(pool) <= 4:
        raise ValueError(f"{fn}: {name} must be one to four tensors")
    n_slots = None
    for t in pool:
        if not isinstance(t, torch.Tensor) or t.dim() < 1 or not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must hold contiguous tensors [n_slots, ...]")
        if n_slots is None:
            n_slots = t.shape[0]
        elif t.shape[0] != n_slots:
            raise ValueError(f"{fn}: the planes of {name} must have one number of slots")
    if n_slots < 1 or any(t.numel() == 0 for t in pool):
        raise ValueError(f"{fn}: the planes of {name} must not be empty")
    addresses = (ctypes.c_void_p * len(pool))(*[t.data_ptr() for t in pool])
    sizes = (ctypes.c_int64 * len(pool))(*[t.numel() // n_slots * t.element_size() for t in pool])
    return pool, n_slots, addresses, sizes


def _pool_device(fn, pool, **named):
    return _one_device(fn, **{f"plane {i}": t for i, t in enumerate(pool)}, **named)


def kda_slots_workspace_size(n_slots: int, N: int = 0) -> int:
    return int(load_library().kda_slots_workspace_size(n_slots, N))


def kda_slots_copy(src, dst, src_slots=None, dst_slots=None, stream=None):
    """dst[dst_slots[n]] = src[src_slots[n]] for two pools that do not overlap (each a tensor or a list of
    up to four, slots first; the same sizes per slot), device int32 lists or None (pair n has slot n).
    A source outside its pool gives zeros, a destination outside is skipped, of several pairs with
    one destination the last is taken.  Returns dst."""
    fn = "kda_slots_copy"
    src_, n_src, sa, sb = _planes(fn, "src", src)
    dst_, n_dst, da, db = _planes(fn, "dst", dst)
    if list(sb) != list(db):
        raise ValueError(f"{fn}: src and dst must have the same planes per slot")
    _expect(fn, "src_slots", src_slots, (None,), (torch.int32,))
    _expect(fn, "dst_slots", dst_slots, (None,), (torch.int32,))
    lists = [t.numel() for t in (src_slots, dst_slots) if t is not None]
    if len(lists) == 2 and lists[0] != lists[1]:
        raise ValueError(f"{fn}: src_slots and dst_slots must have one length")
    N = lists[0] if lists else min(n_src, n_dst)
    dev = _pool_device(fn, src_ + dst_, src_slots=src_slots, dst_slots=dst_slots)
    _, sp = _launch_stream(stream, dev)
    _launch(fn, dev, load_library().kda_slots_copy, sa, da, sb, len(src_), _addr(src_slots), _addr(dst_slots),
            N, n_src, n_dst, sp)
    return dst


def _count(fn, refs, slots, stream):
    _required(fn, refs=refs, slots=slots)
    _expect(fn, "refs", refs, (None,), (torch.int32,))
    _expect(fn, "slots", slots, (None,), (torch.int32,))
    dev = _one_device(fn, refs=refs, slots=slots)
    _, sp = _launch_stream(stream, dev)
    _launch(fn, dev, getattr(load_library(), fn), _addr(refs), _addr(slots), slots.numel(), refs.numel(), sp)
    return refs


def kda_slots_retain(refs, slots, stream=None):
    """One more user of every listed slot (device int32) that is in use; refs int32 [n_slots], the users
    of each slot, is updated in place.  Returns refs."""
    return _count("kda_slots_retain", refs, slots, stream)


def kda_slots_release(refs, slots, stream=None):
    """One user less of every listed slot (device int32); a slot without users is free.  Returns refs."""
    return _count("kda_slots_release", refs, slots, stream)


def kda_slots_fork(pool, refs, parents, children=None, workspace=None, stream=None):
    """For each of parents (device int32 [N], or a number: N new sequences) the lowest free slots of the
    pool (a tensor or a list of up to four, slots first), in order, with the parent's contents --
    zeros without a parent, or for one that is free -- and one user in refs (int32 [n_slots], updated
    in place).  Returns children, int32 [N], -1 where no slot was left."""
    fn = "kda_slots_fork"
    pool, n_slots, pa, pb = _planes(fn, "pool", pool)
    new = isinstance(parents, int)
    N = parents if new else None
    if new:
        if not 0 <= N < 1 << 31:
            raise ValueError(f"{fn}: parents must be an int32 tensor or a number from 0 to 2^31 - 1, got {N}")
    else:
        if not isinstance(parents, torch.Tensor):
            raise TypeError(f"{fn}: parents must be an int32 tensor or a number")
        _expect(fn, "parents", parents, (None,), (torch.int32,))
        N = parents.numel()
    _required(fn, refs=refs)
    _expect(fn, "refs", refs, (n_slots,), (torch.int32,))
    _expect(fn, "children", children, (N,), (torch.int32,))
    dev = _pool_device(fn, pool, refs=refs, parents=None if new else parents, children=children,
                       workspace=workspace)
    ts, sp = _launch_stream(stream, dev)
    if children is None:
        children = _alloc(ts, (N,), torch.int32, dev)
    workspace, ws_bytes = _bytes_of(fn, ts, workspace, kda_slots_workspace_size(n_slots, N), dev)
    _launch(fn, dev, load_library().kda_slots_fork, pa, pb, len(pool), _addr(refs),
            None if new else _addr(parents), _addr(children), N, n_slots, _addr(workspace), ws_bytes, sp)
    return children


def kda_slots_compact(pool, refs, table=None, used=None, workspace=None, stream=None):
    """Moves the used slots of the pool together: with U of them, those from U on go to the free ones
    before U, both in order; refs (int32 [n_slots]) goes along, table (int32, slot numbers, or None) is
    rewritten in place, -1 where it named no used slot.  Returns U, an int32 tensor of one element."""
    fn = "kda_slots_compact"
    pool, n_slots, pa, pb = _planes(fn, "pool", pool)
    _required(fn, refs=refs)
    _expect(fn, "refs", refs, (n_slots,), (torch.int32,))
    if table is not None:
        _expect(fn, "table", table, tuple(table.shape) if isinstance(table, torch.Tensor) else (), (torch.int32,))
    _expect(fn, "used", used, (1,), (torch.int32,))
    dev = _pool_device(fn, pool, refs=refs, table=table, used=used, workspace=workspace)
    ts, sp = _launch_stream(stream, dev)
    if used is None:
        used = _alloc(ts, (1,), torch.int32, dev)
    workspace, ws_bytes = _bytes_of(fn, ts, workspace, kda_slots_workspace_size(n_slots), dev)
    _launch(fn, dev, load_library().kda_slots_compact, pa, pb, len(pool), _addr(refs), _addr(table),
            0 if table is None else table.numel(), _addr(used), n_slots, _addr(workspace), ws_bytes, sp)
    return used
