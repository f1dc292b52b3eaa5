"""Python binding for libkda, the MI355X-native Kimi Delta Attention operator.

Argument marshalling only: every step of the operator runs in the HIP kernels of
``libkda.so`` (built by ``gated_delta_rule_07_amd.build``), called through its C
ABI (``include/kda.h``).  PyTorch supplies device memory and the current HIP
stream; nothing here computes any part of the recurrence, and there is no CPU
fallback: if the library is missing the calls raise.
"""
from __future__ import annotations

import ctypes
from pathlib import Path

import torch

__all__ = ["kda_chunk_fwd", "kda_chunk_fwd_snapshots", "kda_chunk_fwd_varlen", "kda_chunk_fwd_gated",
           "kda_chunk_fwd_split", "kda_chunk_fwd_split_plan", "kda_chunk_fwd_run_chunk",
           "kda_chunk_fwd_split_noalloc", "KDA_SPLIT_SCRATCH_BYTES",
           "kda_decode_step", "kda_decode_step_gated",
           "kda_decode_verify",
           "kda_decode_commit",
           "kda_qk_norm", "kda_cache_fork", "kda_cache_free", "kda_cache_compact", "kda_cache_copy",
           "kda_decode_step_paged", "kda_tree_verify", "kda_tree_commit",
           "kda_status_string", "kda_version",
           "kda_last_hip_error", "library_path", "load_library", "bind", "KdaError",
           "KDA_F32", "KDA_BF16", "KDA_MAX_SNAPSHOTS", "KDA_MAX_DRAFT", "KDA_MAX_PAGES", "KDA_MAX_FORKS",
           "KDA_MAX_PAGED_SEQS", "KDA_MAX_TREE"]

KDA_F32, KDA_BF16 = 0, 1
KDA_MAX_SNAPSHOTS = 128
KDA_MAX_DRAFT = 16
KDA_SPLIT_SCRATCH_BYTES = 64 << 20
KDA_MAX_PAGES = 65536
KDA_MAX_FORKS = 1024
KDA_MAX_PAGED_SEQS = 4096
KDA_MAX_TREE = 64
_PKG = Path(__file__).resolve().parent
_LIB_PATH = _PKG / "libkda.so"
_lib = None


class KdaError(RuntimeError):
    """A libkda call returned a non-OK status."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {kda_status_string(status)}")


def library_path() -> Path:
    return _LIB_PATH


def load_library():
    """Load libkda.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not _LIB_PATH.exists():
        raise RuntimeError(f"libkda is not built ({_LIB_PATH} missing); run "
                           "`python -m gated_delta_rule_07_amd.build` first")
    _lib = bind(_LIB_PATH)
    return _lib


def bind(path) -> ctypes.CDLL:
    """Open a build of the C ABI at `path` and declare its argument types."""
    lib = ctypes.CDLL(str(path))
    vp, i32 = ctypes.c_void_p, ctypes.c_int
    lib.kda_chunk_fwd.restype = i32
    lib.kda_chunk_fwd.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, vp,
                                  i32, i32, i32, i32, i32, i32, vp]
    lib.kda_chunk_fwd_snapshots.restype = i32
    lib.kda_chunk_fwd_snapshots.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, vp, vp, i32, vp,
                                            i32, i32, i32, i32, i32, i32, vp]
    lib.kda_decode_step.restype = i32
    lib.kda_decode_step.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
    lib.kda_chunk_fwd_varlen.restype = i32
    lib.kda_chunk_fwd_varlen.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, vp, vp, i32, i32,
                                         i32, i32, i32, i32, vp]
    lib.kda_chunk_fwd_gated.restype = i32
    lib.kda_chunk_fwd_gated.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, vp,
                                        i32, i32, i32, i32, i32, i32, vp]
    sz = ctypes.c_size_t
    lib.kda_chunk_fwd_split_plan.restype = i32
    lib.kda_chunk_fwd_split_plan.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32,
                                             ctypes.POINTER(i32), ctypes.POINTER(sz)]
    lib.kda_chunk_fwd_split.restype = i32
    lib.kda_chunk_fwd_split.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, vp,
                                        i32, i32, i32, i32, i32, i32, i32, i32, vp, sz, vp]
    lib.kda_chunk_fwd_split_noalloc.restype = i32
    lib.kda_chunk_fwd_split_noalloc.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, vp,
                                                i32, i32, i32, i32, i32, i32, i32, i32, vp]
    lib.kda_decode_step_gated.restype = i32
    lib.kda_decode_step_gated.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
    lib.kda_decode_verify.restype = i32
    lib.kda_decode_verify.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, vp]
    lib.kda_decode_commit.restype = i32
    lib.kda_decode_commit.argtypes = [vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
    i64, f32 = ctypes.c_longlong, ctypes.c_float
    lib.kda_qk_norm.restype = i32
    lib.kda_qk_norm.argtypes = [vp, i64, vp, i64, i32, i32, vp, vp, f32, f32, vp, vp, i32, i32, vp, i64, vp, i64,
                                i32, i32, i32, i32, i32, vp]
    lib.kda_cache_fork.restype = i32
    lib.kda_cache_fork.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
    lib.kda_cache_free.restype = i32
    lib.kda_cache_free.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp]
    lib.kda_cache_compact.restype = i32
    lib.kda_cache_compact.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp]
    lib.kda_cache_copy.restype = i32
    lib.kda_cache_copy.argtypes = [vp, vp, sz, i32, i32, i32, vp, vp, i32, vp]
    lib.kda_decode_step_paged.restype = i32
    lib.kda_decode_step_paged.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, i32,
                                          i32, i32, i32, i32, vp]
    lib.kda_tree_verify.restype = i32
    lib.kda_tree_verify.argtypes = [vp, vp, vp, i32, vp, vp, vp, i32, vp, vp, vp, vp, i32, vp,
                                    i32, i32, i32, i32, i32, vp]
    lib.kda_tree_commit.restype = i32
    lib.kda_tree_commit.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, vp]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_status_string.argtypes = [i32]
    lib.kda_last_hip_error.restype = i32
    lib.kda_last_hip_error.argtypes = []
    lib.kda_version.restype = i32
    lib.kda_version.argtypes = []
    lib.kda_chunk_fwd_run_chunk.restype = i32
    lib.kda_chunk_fwd_run_chunk.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(i32)]
    return lib


def kda_chunk_fwd_run_chunk(qkv_dtype, H, d_k, d_v, chunk: int = 64) -> int:
    """Tokens per chunk a ``kda_chunk_fwd`` call with these sizes runs."""
    code = KDA_BF16 if qkv_dtype == torch.bfloat16 else KDA_F32 if qkv_dtype == torch.float32 else -1
    run = ctypes.c_int(0)
    st = load_library().kda_chunk_fwd_run_chunk(code, int(H), int(d_k), int(d_v), int(chunk), ctypes.byref(run))
    if st != 0:
        raise KdaError(st, "kda_chunk_fwd_run_chunk")
    return run.value


def kda_status_string(status: int) -> str:
    return load_library().kda_status_string(int(status)).decode()


def kda_version() -> int:
    return load_library().kda_version()


def kda_last_hip_error() -> int:
    return load_library().kda_last_hip_error()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"libkda: q/k/v must be bfloat16 or float32, got {t.dtype}")


def _check(t: torch.Tensor, name: str, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"libkda: {name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"libkda: {name} must be on a HIP device, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"libkda: {name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"libkda: {name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"libkda: {name} must be {dtype}, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _prefill_prep(q, k, v, alpha, beta, S0, o, S_T, o_dtype, want_state):
    _check(q, "q")
    dev = q.device
    for t, n in ((k, "k"), (v, "v")):
        _check(t, n, q.dtype, dev)
    if alpha is not None:  # None: the gated call, which checks z and A itself
        _check(alpha, "alpha", torch.float32, dev)
    _check(beta, "beta", torch.float32, dev)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("libkda: q/k/v must be [B,T,H,d]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if (k.shape != q.shape or (alpha is not None and alpha.shape != q.shape) or v.shape[:3] != q.shape[:3]
            or beta.shape != (B, T, H)):
        raise ValueError("libkda: inconsistent shapes")
    if S0 is not None:
        _check(S0, "S0", torch.float32, dev)
        if S0.shape != (B, H, dk, dv):
            raise ValueError("libkda: S0 must be [B,H,d_k,d_v]")
    if o is None:
        o = torch.empty(B, T, H, dv, device=dev, dtype=o_dtype)
    else:
        _check(o, "o", None, dev)
        if o.shape != (B, T, H, dv):
            raise ValueError("libkda: o must be [B,T,H,d_v]")
    if want_state and S_T is None:
        S_T = torch.empty(B, H, dk, dv, device=dev, dtype=torch.float32)
    elif S_T is not None:
        _check(S_T, "S_T", torch.float32, dev)
        if S_T.shape != (B, H, dk, dv):
            raise ValueError("libkda: S_T must be [B,H,d_k,d_v]")
    return dev, (B, T, H, dk, dv), o, S_T


def kda_chunk_fwd(q, k, v, alpha, beta, S0=None, *, chunk: int = 64, o=None, S_T=None,
                  o_dtype=torch.float32, want_state: bool = True, stream=None):
    """Prefill: returns ``(o, S_T)`` (``S_T`` is None when ``want_state`` is False).

    q, k: [B,T,H,d_k]; v: [B,T,H,d_v] (bf16 or fp32, same dtype); alpha: [B,T,H,d_k]
    fp32; beta: [B,T,H] fp32; S0: [B,H,d_k,d_v] fp32 or None (zeros).  ``o`` is
    float32 (default) or bfloat16 (``o_dtype``, or the dtype of a preallocated
    ``o``).  ``S_T`` may be preallocated (it may be ``S0`` for an in-place update).
    """
    lib = load_library()
    dev, (B, T, H, dk, dv), o, S_T = _prefill_prep(q, k, v, alpha, beta, S0, o, S_T, o_dtype, want_state)
    st = lib.kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(alpha), _ptr(beta),
                           _ptr(S0), _ptr(o), _dtype_code(o), _ptr(S_T), B, T, H, dk, dv, int(chunk),
                           _stream(dev, stream))
    if st != 0:
        raise KdaError(st, "kda_chunk_fwd")
    return o, S_T


def kda_chunk_fwd_snapshots(q, k, v, alpha, beta, S0=None, *, snap_tokens, chunk: int = 64, o=None,
                            S_T=None, snaps=None, o_dtype=torch.float32, want_state: bool = True,
                            stream=None):
    """Prefill that also records the state after each count in ``snap_tokens``.

    Returns ``(o, S_T, snaps)`` with ``snaps`` [B,H,len(snap_tokens),d_k,d_v] fp32:
    ``snaps[:, :, j]`` is the state after the first ``snap_tokens[j]`` tokens.  The
    counts must be strictly increasing, in [1, T], and multiples of ``chunk`` (or T);
    at most ``KDA_MAX_SNAPSHOTS`` of them.  Other arguments as ``kda_chunk_fwd``.
    """
    lib = load_library()
    dev, (B, T, H, dk, dv), o, S_T = _prefill_prep(q, k, v, alpha, beta, S0, o, S_T, o_dtype, want_state)
    pos = [int(t) for t in snap_tokens]
    n = len(pos)
    if snaps is None:
        snaps = torch.empty(B, H, n, dk, dv, device=dev, dtype=torch.float32)
    else:
        _check(snaps, "snaps", torch.float32, dev)
        if snaps.shape != (B, H, n, dk, dv):
            raise ValueError("libkda: snaps must be [B,H,n_snap,d_k,d_v]")
    arr = (ctypes.c_int * max(n, 1))(*pos)
    st = lib.kda_chunk_fwd_snapshots(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(alpha), _ptr(beta),
                                     _ptr(S0), _ptr(o), _dtype_code(o), _ptr(S_T), arr, n,
                                     _ptr(snaps) if n > 0 else None, B, T, H, dk, dv, int(chunk),
                                     _stream(dev, stream))
    if st != 0:
        raise KdaError(st, "kda_chunk_fwd_snapshots")
    return o, S_T, snaps


def kda_chunk_fwd_varlen(q, k, v, alpha, beta, cu_seqlens, S0=None, *, chunk: int = 64, o=None, S_T=None,
                         o_dtype=torch.float32, want_state: bool = True, stream=None):
    """Prefill over a packed batch: returns ``(o, S_T)``.

    q, k, alpha: [total_T,H,d_k]; v: [total_T,H,d_v]; beta: [total_T,H];
    cu_seqlens: int32 [N+1] on the device (sequence b is rows cu[b]..cu[b+1]);
    S0: [N,H,d_k,d_v] fp32 or None.  o: [total_T,H,d_v]; S_T: [N,H,d_k,d_v].
    """
    lib = load_library()
    _check(cu_seqlens, "cu_seqlens", torch.int32, q.device if isinstance(q, torch.Tensor) else None)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("libkda: cu_seqlens must be [N+1] with N >= 1")
    N = cu_seqlens.numel() - 1
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("libkda: packed q/k/v must be [total_T,H,d]")
    if S0 is not None and S0.shape[0] != N:
        raise ValueError("libkda: S0 must be [N,H,d_k,d_v]")
    if S_T is not None and S_T.shape[0] != N:
        raise ValueError("libkda: S_T must be [N,H,d_k,d_v]")
    # the packed rows are one [1,total_T,...] batch for the shared checks
    dev, (_, T, H, dk, dv), o4, _ = _prefill_prep(q[None], k[None], v[None], alpha[None], beta[None], None,
                                                  None if o is None else o[None], None, o_dtype, False)
    if S0 is not None:
        _check(S0, "S0", torch.float32, dev)
        if S0.shape != (N, H, dk, dv):
            raise ValueError("libkda: S0 must be [N,H,d_k,d_v]")
    if want_state and S_T is None:
        S_T = torch.empty(N, H, dk, dv, device=dev, dtype=torch.float32)
    elif S_T is not None:
        _check(S_T, "S_T", torch.float32, dev)
        if S_T.shape != (N, H, dk, dv):
            raise ValueError("libkda: S_T must be [N,H,d_k,d_v]")
    st = lib.kda_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(alpha), _ptr(beta), _ptr(S0),
                                  _ptr(o4), _dtype_code(o4), _ptr(S_T), _ptr(cu_seqlens), N, T, H, dk, dv,
                                  int(chunk), _stream(dev, stream))
    if st != 0:
        raise KdaError(st, "kda_chunk_fwd_varlen")
    return o4[0], S_T


def kda_chunk_fwd_gated(q, k, v, z, A, beta, S0=None, *, chunk: int = 64, o=None, S_T=None,
                        o_dtype=torch.float32, want_state: bool = True, stream=None):
    """Prefill with the gate fused in: alpha = exp(-5 sigmoid(e^A z)) is formed in
    the kernels.  z: [B,T,H,d_k] in q's dtype; A: [H] fp32.  Returns ``(o, S_T)``;
    other arguments as ``kda_chunk_fwd``."""
    lib = load_library()
    dev, (B, T, H, dk, dv), o, S_T = _prefill_prep(q, k, v, None, beta, S0, o, S_T, o_dtype, want_state)
    _check(z, "z", q.dtype, dev)
    _check(A, "A", torch.float32, dev)
    if z.shape != q.shape or A.shape != (H,):
        raise ValueError("libkda: z must be shaped like q and A must be [H]")
    st = lib.kda_chunk_fwd_gated(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(z), _ptr(A), _ptr(beta),
                                 _ptr(S0), _ptr(o), _dtype_code(o), _ptr(S_T), B, T, H, dk, dv, int(chunk),
                                 _stream(dev, stream))
    if st != 0:
        raise KdaError(st, "kda_chunk_fwd_gated")
    return o, S_T


def kda_chunk_fwd_split_plan(qkv_dtype, B, T, H, d_k, d_v, *, chunk: int = 64, parts: int = 0,
                             num_cus: int = 0):
    """``(parts, workspace_bytes)`` a split prefill of this shape would use
    (``parts`` 0: the library's choice for ``num_cus`` compute units, 0: the
    current device's)."""
    lib = load_library()
    code = KDA_BF16 if qkv_dtype == torch.bfloat16 else KDA_F32 if qkv_dtype == torch.float32 else -1
    n, ws = ctypes.c_int(0), ctypes.c_size_t(0)
    st = lib.kda_chunk_fwd_split_plan(code, B, T, H, d_k, d_v, int(chunk), int(parts), int(num_cus),
                                      ctypes.byref(n), ctypes.byref(ws))
    if st != 0:
        raise KdaError(st, "kda_chunk_fwd_split_plan")
    return n.value, ws.value


def kda_chunk_fwd_split(q, k, v, alpha, beta, S0=None, *, parts: int = 0, num_cus: int = 0, chunk: int = 64,
                        o=None, S_T=None, workspace=None, o_dtype=torch.float32, want_state: bool = True,
                        stream=None):
    """Prefill with every sequence split into parts that run side by side (a
    two-level scan over the parts).  ``parts`` 0: the library's choice; the
    workspace (a uint8 device tensor) is allocated here when not given.  Returns
    ``(o, S_T)``; other arguments as ``kda_chunk_fwd``."""
    lib = load_library()
    dev, (B, T, H, dk, dv), o, S_T = _prefill_prep(q, k, v, alpha, beta, S0, o, S_T, o_dtype, want_state)
    n, need = kda_chunk_fwd_split_plan(q.dtype, B, T, H, dk, dv, chunk=chunk, parts=parts, num_cus=num_cus)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8, dev)
    st = lib.kda_chunk_fwd_split(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(alpha), _ptr(beta),
                                 _ptr(S0), _ptr(o), _dtype_code(o), _ptr(S_T), B, T, H, dk, dv, int(chunk),
                                 n, 0, _ptr(workspace), workspace.numel() if workspace is not None else 0,
                                 _stream(dev, stream))
    if st != 0:
        raise KdaError(st, "kda_chunk_fwd_split")
    return o, S_T


def kda_chunk_fwd_split_noalloc(q, k, v, alpha, beta, S0=None, *, parts: int = 0, num_cus: int = 0,
                                chunk: int = 64, o=None, S_T=None, o_dtype=torch.float32, want_state: bool = True,
                                stream=None):
    """The split prefill with its workspace in the library's fixed per-GPU scratch
    array (``KDA_SPLIT_SCRATCH_BYTES``): the C call allocates nothing.  Pass
    preallocated ``o`` and ``S_T`` to keep this wrapper from allocating them.
    Calls that overlap on one GPU race.  Returns ``(o, S_T)``; other arguments as
    ``kda_chunk_fwd_split``."""
    lib = load_library()
    dev, (B, T, H, dk, dv), o, S_T = _prefill_prep(q, k, v, alpha, beta, S0, o, S_T, o_dtype, want_state)
    st = lib.kda_chunk_fwd_split_noalloc(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(alpha), _ptr(beta),
                                         _ptr(S0), _ptr(o), _dtype_code(o), _ptr(S_T), B, T, H, dk, dv, int(chunk),
                                         int(parts), int(num_cus), _stream(dev, stream))
    if st != 0:
        raise KdaError(st, "kda_chunk_fwd_split_noalloc")
    return o, S_T


def kda_decode_step_gated(q, k, v, z, A, beta, S, *, o=None, o_dtype=torch.float32, stream=None):
    """Decode with the gate fused in.  z: [B,H,d_k] in q's dtype; A: [H] fp32; the
    rest as ``kda_decode_step``.  Returns ``o``."""
    lib = load_library()
    _check(q, "q")
    dev = q.device
    for t, n in ((k, "k"), (v, "v"), (z, "z")):
        _check(t, n, q.dtype, dev)
    _check(A, "A", torch.float32, dev)
    _check(beta, "beta", torch.float32, dev)
    _check(S, "S", torch.float32, dev)
    if q.dim() != 3:
        raise ValueError("libkda: decode q/k/v must be [B,H,d]")
    B, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or z.shape != q.shape or v.shape[:2] != (B, H) or beta.shape != (B, H) or A.shape != (H,):
        raise ValueError("libkda: inconsistent shapes")
    if S.shape != (B, H, dk, dv):
        raise ValueError("libkda: S must be [B,H,d_k,d_v]")
    if o is None:
        o = torch.empty(B, H, dv, device=dev, dtype=o_dtype)
    else:
        _check(o, "o", None, dev)
        if o.shape != (B, H, dv):
            raise ValueError("libkda: o must be [B,H,d_v]")
    st = lib.kda_decode_step_gated(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(z), _ptr(A), _ptr(beta),
                                   _ptr(S), _ptr(o), _dtype_code(o), B, H, dk, dv, _stream(dev, stream))
    if st != 0:
        raise KdaError(st, "kda_decode_step_gated")
    return o


def kda_decode_step(q, k, v, alpha, beta, S, *, o=None, o_dtype=torch.float32, stream=None):
    """Decode one token per (sequence, head); ``S`` ([B,H,d_k,d_v] fp32) is updated
    in place.  q, k: [B,H,d_k]; v: [B,H,d_v]; alpha: [B,H,d_k]; beta: [B,H].
    Returns ``o`` ([B,H,d_v], float32 by default or bfloat16)."""
    lib = load_library()
    _check(q, "q")
    dev = q.device
    for t, n in ((k, "k"), (v, "v")):
        _check(t, n, q.dtype, dev)
    _check(alpha, "alpha", torch.float32, dev)
    _check(beta, "beta", torch.float32, dev)
    _check(S, "S", torch.float32, dev)
    if q.dim() != 3:
        raise ValueError("libkda: decode q/k/v must be [B,H,d]")
    B, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or alpha.shape != q.shape or v.shape[:2] != (B, H) or beta.shape != (B, H):
        raise ValueError("libkda: inconsistent shapes")
    if S.shape != (B, H, dk, dv):
        raise ValueError("libkda: S must be [B,H,d_k,d_v]")
    if o is None:
        o = torch.empty(B, H, dv, device=dev, dtype=o_dtype)
    else:
        _check(o, "o", None, dev)
        if o.shape != (B, H, dv):
            raise ValueError("libkda: o must be [B,H,d_v]")
    st = lib.kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(alpha), _ptr(beta),
                             _ptr(S), _ptr(o), _dtype_code(o), B, H, dk, dv, _stream(dev, stream))
    if st != 0:
        raise KdaError(st, "kda_decode_step")
    return o


def kda_decode_verify(q, k, v, alpha, beta, S, *, o=None, u=None, o_dtype=torch.float32, stream=None):
    """Speculative decoding, pass 1: apply K draft tokens per (sequence, head)
    without changing ``S``.  q, k: [B,K,H,d_k]; v: [B,K,H,d_v]; alpha: [B,K,H,d_k];
    beta: [B,K,H]; S: [B,H,d_k,d_v] fp32 (read only).  Returns ``(o, u)``: o
    [B,K,H,d_v] (o_t as if the first t drafts were accepted) and u [B,H,K,d_v]
    fp32, the write vectors ``kda_decode_commit`` needs."""
    lib = load_library()
    _check(q, "q")
    dev = q.device
    for t, n in ((k, "k"), (v, "v")):
        _check(t, n, q.dtype, dev)
    _check(alpha, "alpha", torch.float32, dev)
    _check(beta, "beta", torch.float32, dev)
    _check(S, "S", torch.float32, dev)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("libkda: draft q/k/v must be [B,K,H,d]")
    B, K, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or alpha.shape != q.shape or v.shape[:3] != q.shape[:3] or beta.shape != (B, K, H):
        raise ValueError("libkda: inconsistent shapes")
    if S.shape != (B, H, dk, dv):
        raise ValueError("libkda: S must be [B,H,d_k,d_v]")
    if o is None:
        o = torch.empty(B, K, H, dv, device=dev, dtype=o_dtype)
    else:
        _check(o, "o", None, dev)
        if o.shape != (B, K, H, dv):
            raise ValueError("libkda: o must be [B,K,H,d_v]")
    if u is None:
        u = torch.empty(B, H, K, dv, device=dev, dtype=torch.float32)
    else:
        _check(u, "u", torch.float32, dev)
        if u.shape != (B, H, K, dv):
            raise ValueError("libkda: u must be [B,H,K,d_v]")
    st = lib.kda_decode_verify(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(alpha), _ptr(beta), _ptr(S),
                               _ptr(o), _dtype_code(o), _ptr(u), B, K, H, dk, dv, _stream(dev, stream))
    if st != 0:
        raise KdaError(st, "kda_decode_verify")
    return o, u


def kda_decode_commit(k, alpha, u, n_accept, S, *, stream=None):
    """Speculative decoding, pass 2: advance ``S`` in place over the accepted
    drafts, ``n_accept[b]`` of them for sequence b (int32 [B] on the device,
    clamped to [0, K]).  k, alpha: the drafts' [B,K,H,d_k] inputs of
    ``kda_decode_verify``; u: its [B,H,K,d_v] output.  Returns ``S``."""
    lib = load_library()
    _check(k, "k")
    dev = k.device
    _check(alpha, "alpha", torch.float32, dev)
    _check(u, "u", torch.float32, dev)
    _check(n_accept, "n_accept", torch.int32, dev)
    _check(S, "S", torch.float32, dev)
    if k.dim() != 4:
        raise ValueError("libkda: draft k must be [B,K,H,d_k]")
    B, K, H, dk = k.shape
    dv = S.shape[-1]
    if alpha.shape != k.shape or S.shape != (B, H, dk, dv) or u.shape != (B, H, K, dv) or n_accept.shape != (B,):
        raise ValueError("libkda: inconsistent shapes")
    st = lib.kda_decode_commit(_ptr(k), _dtype_code(k), _ptr(alpha), _ptr(u), _ptr(n_accept), _ptr(S),
                               B, K, H, dk, dv, _stream(dev, stream))
    if st != 0:
        raise KdaError(st, "kda_decode_commit")
    return S


_NORMS = {"l2": 0, "rms": 1}
_PAIRINGS = {"halves": 0, "pairs": 1}
_CODES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}
_I32, _F32 = torch.int32, torch.float32

# The calls below serve single tokens too, where a step's time is the time to issue
# it: their checks read each property of a tensor once, and say what is wrong with
# it only when something is.


def _raw_stream(index):
    """The current stream of device `index`, as the pointer the C ABI takes."""
    return torch.cuda.current_stream(index).cuda_stream


_current_device = torch.cuda.current_device
if hasattr(torch._C, "_cuda_getCurrentRawStream") and hasattr(torch._C, "_cuda_getDevice"):
    # the same without a Stream object, and without asking whether HIP is set up (a tensor is there)
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice  # noqa: F811


def _run(name, index, stream, *args):
    """Call `name` of the library on device `index` (made current for the call where it is not)."""
    fn = getattr(_lib or load_library(), name)
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == _current_device():
        st = fn(*args, s)
    else:
        with torch.cuda.device(index):
            st = fn(*args, s)
    if st != 0:
        raise KdaError(st, name)


def _tensor(t, name):
    """t, which has to be a tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"libkda: {name} must be a torch.Tensor")
    return t


def _device_of(t, name):
    """The index of t's device; t has to be a tensor on a HIP device."""
    _tensor(t, name)
    if not t.is_cuda:
        raise ValueError(f"libkda: {name} must be on a HIP device, got {t.device}")
    return t.get_device()


def _need_in_words(t, name, dtype, index, shape):
    """The address of t, which has to be a dense tensor of this dtype and shape on device `index`."""
    _check(t, name, dtype, torch.device("cuda", index))
    if t.shape != shape:
        raise ValueError(f"libkda: {name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _argument_forms():
    """(_need, _rows): one compiled call each, or Python forms of the same where the helper is missing, or was built
    against another PyTorch than this one (it reads the layout of its objects): only the time of a call grows."""
    try:
        from . import _kda_args
        if _kda_args.torch_version == torch.__version__:
            _kda_args.set_refuse(_need_in_words)
            return _kda_args.need, _kda_args.rows
    except (ImportError, AttributeError):
        pass
    return _need_in_words, lambda t, dtype, index: None


_need, _rows = _argument_forms()


def _may(t, name, dtype, index, shape):
    return None if t is None else _need(t, name, dtype, index, shape)


def _filled(shape, dtype, device, value, stream):
    """A new tensor for a call that may pass over some of its rows: `value` throughout, filled on the call's stream."""
    if stream is None:
        return torch.full(shape, value, dtype=dtype, device=device)
    t = torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return t.fill_(value)


def _io_code(t, name):
    """kda_dtype of a bf16 or fp32 tensor."""
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"libkda: {name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _head_rows(t, name, dtype, index):
    """(address, tokens, heads, d, row stride in elements) of [n,H,d] or [B,T,H,d] rows of dense heads."""
    got = _rows(t, dtype, index)
    if got is not None:
        return got
    if _device_of(t, name) != index or t.dtype != dtype:
        raise ValueError(f"libkda: {name} must be {dtype} on device {index}, got {t.dtype} on {t.device}")
    shape, st = t.shape, t.stride()
    if len(shape) == 3:
        n, H, d = shape
        row = st[0]
    elif len(shape) == 4:
        B, T, H, d = shape
        n, row = B * T, st[1] if T > 1 else st[0]
        if B > 1 and T > 1 and st[0] != T * row:
            raise ValueError(f"libkda: the token rows of {name} must be evenly spaced")
    else:
        raise ValueError(f"libkda: {name} must be [n,H,d] or [B,T,H,d]")
    if n and ((st[-1] != 1 and d > 1) or (st[-2] != d and H > 1)):
        raise ValueError(f"libkda: the heads of a token of {name} must be dense")
    return t.data_ptr(), n, H, d, row


def kda_qk_norm(q, k=None, *, norm: str = "l2", q_weight=None, k_weight=None, eps: float = 1e-6, q_scale: float = 1.0,
                positions=None, inv_freq=None, pairing: str = "halves", q_out=None, k_out=None, out_dtype=None,
                stream=None):
    """Queries and keys normalised for each head, and rotated by position: ``(q_out, k_out)``.

    q: [n,H_q,d] or [B,T,H_q,d], k: the same with H_k heads, or None (bf16 or fp32, same dtype; token rows
    may be slices of wider rows, the heads of a token are dense).  ``norm``: "l2" divides by
    sqrt(sum x^2 + eps), "rms" by sqrt(mean x^2 + eps); ``q_weight``, ``k_weight``: [d] fp32 factors.  With
    ``inv_freq`` ([rot/2] fp32) the first rot values of each head turn by ``positions`` (one int32 per token) times
    inv_freq, in pairs (i, i + rot/2) ("halves") or (2i, 2i + 1) ("pairs").  Queries are multiplied by ``q_scale``
    at the end.  The outputs are dense in ``out_dtype`` (the inputs' by default) unless given; each may be its
    input."""
    dev = _device_of(q, "q")
    dt = q.dtype
    code = _io_code(q, "q")
    qp, n, Hq, d, qs = _head_rows(q, "q", dt, dev)
    nm, pr = _NORMS.get(norm), _PAIRINGS.get(pairing)
    if nm is None or pr is None:
        raise ValueError('libkda: norm is "l2" or "rms", pairing "halves" or "pairs"')
    kp, Hk, ks = None, 0, 0
    if k is not None:
        kp, nk, Hk, dk, ks = _head_rows(k, "k", dt, dev)
        if nk != n or dk != d or k.dim() != q.dim() or (q.dim() == 4 and k.shape[:2] != q.shape[:2]):
            raise ValueError("libkda: q and k must agree in tokens and head size")
    qw = None if q_weight is None else _need(q_weight, "q_weight", _F32, dev, (d,))
    kw = None if k_weight is None else _need(k_weight, "k_weight", _F32, dev, (d,))
    rot, pos, freq = 0, None, None
    if inv_freq is not None and _tensor(inv_freq, "inv_freq").numel():
        rot = 2 * inv_freq.numel()
        freq = _need(inv_freq, "inv_freq", _F32, dev, (rot // 2,))
        if positions is None:
            raise ValueError("libkda: a rotation needs positions")
        pos = _need(positions, "positions", _I32, dev, _tensor(positions, "positions").shape)
        if positions.numel() != n or (q.dim() == 4 and positions.dim() > 1 and positions.shape != q.shape[:2]):
            raise ValueError("libkda: positions must have one entry per token")
    if out_dtype is None:
        out_dtype = dt if q_out is None else _tensor(q_out, "q_out").dtype
    out_code = _CODES.get(out_dtype)
    if out_code is None:
        raise TypeError(f"libkda: outputs must be bfloat16 or float32, got {out_dtype}")
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    qop, qos = _head_out(q_out, "q_out", q, dev, out_dtype)
    kop, kos = None, 0
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=out_dtype, device=k.device)
        kop, kos = _head_out(k_out, "k_out", k, dev, out_dtype)
    elif k_out is not None:
        raise ValueError("libkda: k_out without k")
    _run("kda_qk_norm", dev, stream, qp, qs, kp, ks, code, nm, qw, kw, eps, q_scale, pos, freq, rot, pr,
         qop, qos, kop, kos, out_code, n, Hq, Hk, d)
    return q_out, k_out


def _head_out(o, name, x, dev, dtype):
    """(address, row stride) of an output of kda_qk_norm for the input x."""
    op, _, _, _, row = _head_rows(o, name, dtype, dev)
    if o.shape != x.shape:
        raise ValueError(f"libkda: {name} must be shaped like its input")
    return op, row


def _table(table, ref):
    """(device, n_rows, width, n_pages, addresses of table and ref)."""
    dev = _device_of(table, "table")
    if table.dim() != 2 or not isinstance(ref, torch.Tensor) or ref.dim() != 1:
        raise ValueError("libkda: table must be [n_rows,width] and ref [n_pages]")
    R, W = table.shape
    P = ref.shape[0]
    return dev, R, W, P, _need(table, "table", _I32, dev, (R, W)), _need(ref, "ref", _I32, dev, (P,))


def _move_list(moves, n_moves, room, t, stream):
    """moves (pairs of -1) and n_moves, made on t's device where they are not given, and their addresses."""
    dev = t.get_device()
    if moves is None:
        moves = _filled((max(room, 1), 2), _I32, t.device, -1, stream)
    if n_moves is None:
        n_moves = torch.empty(1, dtype=_I32, device=t.device)
    rows = moves.shape[0] if _tensor(moves, "moves").dim() == 2 else 0
    mp, np_ = _need(moves, "moves", _I32, dev, (max(rows, room), 2)), _need(n_moves, "n_moves", _I32, dev, (1,))
    return moves, n_moves, mp, np_


def kda_cache_fork(table, ref, parents, children, n_private: int = 1, *, moves=None, n_moves=None, stream=None):
    """Rows ``children`` of the page table become copies of rows ``parents`` (-1: empty rows), in place: the
    first ``n_private`` entries on free pages of their own, the others shared.  Returns ``(moves, n_moves)``, the
    page copies that ``kda_cache_copy`` has to carry out on each pool (a list that the call makes itself holds pairs of -1,
    which are passed over, behind them).  table: [n_rows,width] int32; ref:
    [n_pages] int32; parents, children: [n] int32 on the device.  A fork that cannot be served (no free pages
    left, the child's row in use) leaves the child's row as it was."""
    dev, R, W, P, tp, rp = _table(table, ref)
    n = children.numel() if isinstance(children, torch.Tensor) else -1
    cp, pp = _need(children, "children", _I32, dev, (n,)), _need(parents, "parents", _I32, dev, (n,))
    moves, n_moves, mp, np_ = _move_list(moves, n_moves, n * max(n_private, 0), table, stream)
    _run("kda_cache_fork", dev, stream, tp, rp, pp, cp, mp, np_, n, n_private, R, W, P)
    return moves, n_moves


def kda_cache_free(table, ref, rows, *, stream=None):
    """The rows listed ([n] int32 on the device) hold nothing any more; their pages' refs are counted down."""
    dev, R, W, P, tp, rp = _table(table, ref)
    n = rows.numel() if isinstance(rows, torch.Tensor) else -1
    _run("kda_cache_free", dev, stream, tp, rp, _need(rows, "rows", _I32, dev, (n,)), n, R, W, P)


def kda_cache_compact(table, ref, *, table_out=None, ref_out=None, moves=None, n_moves=None, n_live=None, stream=None):
    """Packs the pages in use into the lowest ones: ``(table_out, ref_out, moves, n_moves, n_live)``.  Pass
    ``table_out=table`` and ``ref_out=ref`` for an update in place; ``moves`` (room for n_pages // 2 pairs) is what
    ``kda_cache_copy`` has to carry out on each pool."""
    dev, R, W, P, tp, rp = _table(table, ref)
    table_out = torch.empty_like(table) if table_out is None else table_out
    ref_out = torch.empty_like(ref) if ref_out is None else ref_out
    n_live = torch.empty(1, dtype=_I32, device=table.device) if n_live is None else n_live
    to, ro = _need(table_out, "table_out", _I32, dev, (R, W)), _need(ref_out, "ref_out", _I32, dev, (P,))
    moves, n_moves, mp, np_ = _move_list(moves, n_moves, max(P // 2, 1), table, stream)
    _run("kda_cache_compact", dev, stream, tp, rp, to, ro, mp, np_, _need(n_live, "n_live", _I32, dev, (1,)), R, W, P)
    return table_out, ref_out, moves, n_moves, n_live


def kda_cache_copy(pool, moves, n_moves=None, *, src=None, n_layers=None, stream=None):
    """Page ``moves[i, 1]`` of ``pool`` becomes a copy of page ``moves[i, 0]`` of ``src`` (default: of the pool
    itself; -1: zeros), for the first ``n_moves`` ([1] int32 on the device; default: all) pairs.  A pool is
    [n_pages, ...], or [n_layers, n_pages, ...] with ``n_layers`` given; any dtype.  Returns ``pool``."""
    dev = _device_of(pool, "pool")
    src = pool if src is None else src
    _device_of(src, "src")
    lead, L = (1, 1) if n_layers is None else (2, n_layers)
    shape, other = pool.shape, src.shape
    if len(shape) < lead or other[lead:] != shape[lead:] or len(other) != len(shape) or (
            lead == 2 and (shape[0] != L or other[0] != L)):
        raise ValueError("libkda: pool and src must be [n_pages,...], or [n_layers,n_pages,...] with n_layers, of one page shape")
    pp, sp = _need(pool, "pool", pool.dtype, dev, shape), _need(src, "src", pool.dtype, dev, other)
    most = moves.shape[0] if isinstance(moves, torch.Tensor) and moves.dim() == 2 else -1
    mp, np_ = _need(moves, "moves", _I32, dev, (most, 2)), _may(n_moves, "n_moves", _I32, dev, (1,))
    page = pool.element_size() * shape[lead:].numel()
    _run("kda_cache_copy", dev, stream, sp, pp, page, L, other[lead - 1], shape[lead - 1], mp, np_, most)
    return pool


def _state_pool(pool, H, dk, dv, dev):
    """(pages, address) of a pool of states."""
    n = pool.shape[0] if isinstance(pool, torch.Tensor) and pool.dim() == 4 else -1
    return n, _need(pool, "pool", _F32, dev, (n, H, dk, dv))


def kda_decode_step_paged(q, k, v, alpha, beta, pool, pages_in, pages_out=None, *, z=None, A=None, o=None,
                          o_dtype=torch.float32, stream=None):
    """Decode one token per (sequence, head) on a pool of state pages: the state on page ``pages_in[b]`` of
    ``pool`` ([n_pages,H,d_k,d_v] fp32) goes to page ``pages_out[b]`` (default: the same page).  ``alpha`` None: the
    gate inputs z and A of ``kda_decode_step_gated``.  A sequence whose page is out of range (padding: -1), or is
    written by another sequence of the call, is passed over: its row of ``o`` and the pool are left as they were.
    Returns ``o``; where it is not given it is made here, with zeros in the rows passed over (a fill that a step with
    its own ``o`` does without)."""
    dev = _device_of(q, "q")
    if q.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("libkda: decode q/k/v must be [B,H,d]")
    shape, dt = q.shape, q.dtype
    B, H, dk = shape
    dv = v.shape[2]
    code = _io_code(q, "q")
    qp, kp, vp = _need(q, "q", dt, dev, shape), _need(k, "k", dt, dev, shape), _need(v, "v", dt, dev, (B, H, dv))
    if alpha is not None:
        if z is not None or A is not None:
            raise ValueError("libkda: give alpha, or z and A")
        ap, zp, Ap = _need(alpha, "alpha", _F32, dev, shape), None, None
    else:
        ap, zp, Ap = None, _need(z, "z", dt, dev, shape), _need(A, "A", _F32, dev, (H,))
    bp = _need(beta, "beta", _F32, dev, (B, H))
    P, poolp = _state_pool(pool, H, dk, dv, dev)
    ip, op = _need(pages_in, "pages_in", _I32, dev, (B,)), _may(pages_out, "pages_out", _I32, dev, (B,))
    if o is None:
        o = _filled((B, H, dv), o_dtype, q.device, 0.0, stream)
    odt = _tensor(o, "o").dtype
    _run("kda_decode_step_paged", dev, stream, qp, kp, vp, code, ap, zp, Ap, bp, poolp, P, ip, op,
         _need(o, "o", odt, dev, (B, H, dv)), _io_code(o, "o"), B, H, dk, dv)
    return o


def kda_tree_verify(q, k, v, alpha, beta, pool, pages, parents, n_nodes=None, *, o=None, u=None, o_dtype=torch.float32,
                    stream=None):
    """Run a tree of drafted tokens against each sequence's state without changing it: ``(o, u)``.

    q, k: [B,K,H,d_k]; v: [B,K,H,d_v]; alpha: [B,K,H,d_k]; beta: [B,K,H]; pool: [n_pages,H,d_k,d_v] fp32, ``pages``
    [B] int32 the page of each sequence (None: page b).  ``parents`` [B,K] int32: the node that node t follows (its
    index is smaller), -1 for the state itself; ``n_nodes`` [B] int32: how many nodes each tree has (None: K).  o:
    [B,K,H,d_v], the output after the path to each node; u: [B,H,K,d_v] fp32, what ``kda_tree_commit`` needs.  Rows
    behind a tree's last node, and those of a sequence whose page is out of range, are left as they were; in an ``o`` or
    ``u`` that is not given, and made here, they are zeros."""
    dev = _device_of(q, "q")
    if q.dim() != 4 or not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("libkda: draft q/k/v must be [B,K,H,d]")
    shape, dt = q.shape, q.dtype
    B, K, H, dk = shape
    dv = v.shape[3]
    code = _io_code(q, "q")
    qp, kp, vp = _need(q, "q", dt, dev, shape), _need(k, "k", dt, dev, shape), _need(v, "v", dt, dev, (B, K, H, dv))
    ap, bp = _need(alpha, "alpha", _F32, dev, shape), _need(beta, "beta", _F32, dev, (B, K, H))
    P, poolp = _state_pool(pool, H, dk, dv, dev)
    pg, pa, nn = _may(pages, "pages", _I32, dev, (B,)), _need(parents, "parents", _I32, dev, (B, K)), _may(n_nodes, "n_nodes", _I32, dev, (B,))
    whole = pages is None and n_nodes is None  # (every row is written)
    if o is None:
        shape = (B, K, H, dv)
        o = torch.empty(shape, device=q.device, dtype=o_dtype) if whole else _filled(shape, o_dtype, q.device, 0.0, stream)
    if u is None:
        shape = (B, H, K, dv)
        u = torch.empty(shape, device=q.device, dtype=_F32) if whole else _filled(shape, _F32, q.device, 0.0, stream)
    odt = _tensor(o, "o").dtype
    _run("kda_tree_verify", dev, stream, qp, kp, vp, code, ap, bp, poolp, P, pg, pa, nn, _need(o, "o", odt, dev, (B, K, H, dv)),
         _io_code(o, "o"), _need(u, "u", _F32, dev, (B, H, K, dv)), B, K, H, dk, dv)
    return o, u


def kda_tree_commit(k, alpha, u, parents, last, pool, pages_in, pages_out=None, n_nodes=None, *, stream=None):
    """Advance each sequence's state over the accepted path of its tree: page ``pages_out[b]`` (default: the same
    page) receives the state after the nodes from the root to ``last[b]`` ([B] int32; out of range: nothing was
    accepted), from the state on page ``pages_in[b]`` (None: page b).  k, alpha, parents, n_nodes: the arguments
    of ``kda_tree_verify``; u: its output.  Pages out of range or shared are treated as
    ``kda_decode_step_paged`` does.  Returns ``pool``."""
    dev = _device_of(k, "k")
    if k.dim() != 4 or not isinstance(u, torch.Tensor) or u.dim() != 4:
        raise ValueError("libkda: draft k must be [B,K,H,d_k] and u [B,H,K,d_v]")
    shape = k.shape
    B, K, H, dk = shape
    dv = u.shape[3]
    code = _io_code(k, "k")
    kp, ap, up = _need(k, "k", k.dtype, dev, shape), _need(alpha, "alpha", _F32, dev, shape), _need(u, "u", _F32, dev, (B, H, K, dv))
    P, poolp = _state_pool(pool, H, dk, dv, dev)
    pa, lp = _need(parents, "parents", _I32, dev, (B, K)), _need(last, "last", _I32, dev, (B,))
    nn, ip, op = (_may(t, name, _I32, dev, (B,)) for t, name in ((n_nodes, "n_nodes"), (pages_in, "pages_in"), (pages_out, "pages_out")))
    _run("kda_tree_commit", dev, stream, kp, code, ap, up, pa, nn, lp, poolp, P, ip, op, B, K, H, dk, dv)
    return pool
