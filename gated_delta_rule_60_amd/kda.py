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
    if path == lib_path():
        _lib = lib
    return lib


EXPORTED = ["kda_status_string", "kda_version", "kda_gate", "kda_chunk_fwd_workspace_size",
            "kda_chunk_fwd", "kda_chunk_fwd_gated", "kda_chunk_fwd_gated_noalloc",
            "kda_chunk_fwd_checkpointed", "kda_decode_step", "kda_decode_verify",
            "kda_decode_commit", "kda_linear_chunk_workspace_size", "kda_linear_chunk_fwd",
            "kda_linear_chunk_bwd", "kda_linear_decode_step", "kda_state_store", "kda_state_load"]

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
    if t.shape == shape and (dtypes is None or t.dtype in dtypes) and t.is_contiguous():
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
