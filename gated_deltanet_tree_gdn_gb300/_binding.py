"""ctypes binding of libgdntree's C ABI (include/gdn_tree.h).

Argument marshalling only: dtype/shape/contiguity checks on torch tensors,
then device pointers and the current CUDA stream go straight to the C entry
points; every step of the computation runs in the library's kernels.  There
is no fallback: if the library is not built, every call raises.

A call runs on torch's current stream, or, with `stream=` (a torch.cuda.Stream or
ExternalStream), as it would under torch.cuda.stream(stream): its inputs must be
ready on that stream, and the tensors that it allocates belong to it.
"""

from __future__ import annotations

import ctypes
import os
from operator import index

import torch

from . import build as _build

BF16, F32 = 0, 1
OK, EINVAL, EUNSUPPORTED, ECUDA = 0, -1, -2, -3
STATUS_OK, STATUS_BAD_TREE, STATUS_BAD_PATH, STATUS_TIMEOUT, STATUS_BAD_LAYOUT = 0, 1, 2, 3, 4

SYMBOLS = ("gdn_tree_verify", "gdn_tree_commit", "gdn_tree_commit_verify",
           "gdn_tree_verify_recurrent", "gdn_tree_verify_packed", "gdn_tree_commit_packed",
           "gdn_tree_commit_verify_packed", "gdn_tree_build_topw", "gdn_tree_prefill", "gdn_tree_prefill_workspace",
           "gdn_tree_decode_step", "gdn_tree_attend", "gdn_tree_attend_workspace",
           "gdn_tree_cache_append", "gdn_tree_norm_rope", "gdn_tree_cache_append_rope",
           "gdn_tree_positions", "gdn_tree_rope_frequencies", "gdn_tree_strerror",
           "gdn_tree_version")


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "N", "Hqk", "Hv", "dk", "dv", "dtype")]


class AttendDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "N", "Hq", "Hkv", "D", "dtype",
                                              "page_size", "n_pages", "table_width",
                                              "prefix_len")]


NORMS = {None: 0, "rms": 1, "unit": 2}
STRETCHES = {None: 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class Rope(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rotary_dim", "interleaved", "norm")] + [
        (n, ctypes.c_float) for n in ("scale", "eps")]


class RopeStretch(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32)] + [
        (n, ctypes.c_double) for n in ("factor", "trained_len", "fast", "slow")]


class Strides(ctypes.Structure):
    _fields_ = [("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class HeadStrides(ctypes.Structure):
    _fields_ = [(n, Strides) for n in ("q", "k", "v", "q_out", "k_out", "v_out")]


class GdnTreeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {strerror(code)} (code {code})")
        self.code = code


_lib = None


def library_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load libgdntree (built by ``build.build_library``); raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB
    if not os.path.exists(p):
        raise RuntimeError(
            f"libgdntree is not built ({p} missing): run "
            "`python -m gated_deltanet_tree_gdn_gb300.build` first")
    lib = ctypes.CDLL(p)
    vp, fp, ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    lib.gdn_tree_verify.argtypes = [vp, vp, vp, fp, fp, ip, fp, vp, fp, Dims, ip, vp]
    lib.gdn_tree_verify.restype = ctypes.c_int
    lib.gdn_tree_verify_recurrent.argtypes = [vp, vp, vp, fp, fp, ip, fp, vp, fp, Dims, ip, vp]
    lib.gdn_tree_verify_recurrent.restype = ctypes.c_int
    lib.gdn_tree_commit.argtypes = [ip, ip, ip, fp, vp, fp, fp, fp, Dims, ctypes.c_int32, ip, vp]
    lib.gdn_tree_commit.restype = ctypes.c_int
    lib.gdn_tree_commit_verify.argtypes = [ip, ip, ip, fp, vp, fp, ctypes.c_int32, ctypes.c_int32,
                                           fp, fp, vp, vp, vp, fp, fp, ip, vp, fp, Dims, ip, ip,
                                           vp]
    lib.gdn_tree_commit_verify.restype = ctypes.c_int
    i32 = ctypes.c_int32
    lib.gdn_tree_verify_packed.argtypes = [vp, vp, vp, fp, fp, ip, ip, i32, fp, ip, i32, vp, fp,
                                           Dims, ip, vp]
    lib.gdn_tree_verify_packed.restype = ctypes.c_int
    lib.gdn_tree_commit_packed.argtypes = [ip, ip, ip, ip, i32, fp, vp, fp, fp, fp, ip, i32, Dims,
                                           i32, ip, vp]
    lib.gdn_tree_commit_packed.restype = ctypes.c_int
    lib.gdn_tree_commit_verify_packed.argtypes = [ip, ip, ip, ip, i32, fp, vp, fp, i32, i32, fp,
                                                  fp, ip, i32, vp, vp, vp, fp, fp, ip, ip, i32,
                                                  vp, fp, Dims, ip, ip, vp]
    lib.gdn_tree_commit_verify_packed.restype = ctypes.c_int
    lib.gdn_tree_build_topw.argtypes = [fp, i32, i32, i32, i32, i32, ip, ip, fp, ip, vp]
    lib.gdn_tree_build_topw.restype = ctypes.c_int
    lib.gdn_tree_prefill.argtypes = [vp, vp, vp, fp, fp, ip, i32, fp, fp, ip, i32, vp, Dims, ip,
                                     vp, ctypes.c_size_t, vp]
    lib.gdn_tree_prefill_workspace.argtypes = [Dims, i32]
    lib.gdn_tree_prefill_workspace.restype = ctypes.c_size_t
    lib.gdn_tree_prefill.restype = ctypes.c_int
    lib.gdn_tree_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, fp, ip, i32, vp, Dims, ip, vp]
    lib.gdn_tree_decode_step.restype = ctypes.c_int
    lib.gdn_tree_attend.argtypes = [vp, vp, vp, ip, ip, vp, vp, ip, ip, ip, ctypes.c_float, vp,
                                    fp, AttendDims, ip, vp, ctypes.c_size_t, vp]
    lib.gdn_tree_attend.restype = ctypes.c_int
    lib.gdn_tree_attend_workspace.argtypes = [AttendDims]
    lib.gdn_tree_attend_workspace.restype = ctypes.c_size_t
    lib.gdn_tree_cache_append.argtypes = [vp, vp, ip, ip, i32, ip, vp, vp, ip, ip, ip, AttendDims,
                                          ip, vp]
    lib.gdn_tree_cache_append.restype = ctypes.c_int
    lib.gdn_tree_norm_rope.argtypes = [vp, vp, ip, vp, fp, fp, vp, vp, HeadStrides, AttendDims,
                                       Rope, vp]
    lib.gdn_tree_norm_rope.restype = ctypes.c_int
    lib.gdn_tree_cache_append_rope.argtypes = [vp, vp, vp, vp, fp, fp, ip, vp, vp, vp, vp, vp, ip,
                                               ip, ip, HeadStrides, AttendDims, Rope, ip, vp]
    lib.gdn_tree_cache_append_rope.restype = ctypes.c_int
    lib.gdn_tree_positions.argtypes = [ip, ip, ip, i32, ip, i32, i32, i32, ip, vp]
    lib.gdn_tree_positions.restype = ctypes.c_int
    lib.gdn_tree_rope_frequencies.argtypes = [i32, ctypes.c_double, RopeStretch, vp, vp]
    lib.gdn_tree_rope_frequencies.restype = ctypes.c_int
    lib.gdn_tree_strerror.argtypes = [ctypes.c_int]
    lib.gdn_tree_strerror.restype = ctypes.c_char_p
    lib.gdn_tree_version.argtypes = []
    lib.gdn_tree_version.restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def strerror(code: int) -> str:
    try:
        return load().gdn_tree_strerror(int(code)).decode()
    except RuntimeError:
        return f"code {code}"


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


# The marshalling below runs on every call, ahead of a launch that can take only a few
# microseconds (a decoding step of one sequence), so it is kept lean: pointers go to
# ctypes as plain integers, shapes are compared as they are, and the stream is read as
# its raw handle.

def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t: torch.Tensor, name: str, dtype=None, shape=None):
    if (type(t) is torch.Tensor and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


# the current stream's handle without building a Stream object (the public call is the
# fallback where the accessor is absent)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream() -> int:
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _on(stream, call, args):
    """The call with these arguments under torch.cuda.stream(stream): what is allocated, copied or
    read on the way then belongs to the stream that the kernels run on.  (A block of the current
    stream could be handed out again, and a copy made, while they run.)"""
    with torch.cuda.stream(stream):
        return call(**dict(args, stream=None))


_dims_cache: dict = {}


def dims_of(q: torch.Tensor, v: torch.Tensor) -> Dims:
    key = (q.shape, v.shape, q.dtype)
    d = _dims_cache.get(key)
    if d is None:
        B, N, Hqk, dk = q.shape
        Hv, dv = v.shape[2], v.shape[3]
        d = Dims(B, N, Hqk, Hv, dk, dv, _dtype_code(q))
        if len(_dims_cache) < 256:
            _dims_cache[key] = d
    return d


def verify(q, k, v, log_alpha, beta, parent, S0, *, o=None, U=None, dev_status=None,
           stream=None):
    """Tree verification (C ABI gdn_tree_verify).  Returns (o, U).

    q, k [B,N,Hqk,dk] and v [B,N,Hv,dv] in bf16 or fp32; log_alpha, beta
    [B,N,Hv] fp32; parent [B,N] int32; S0 [B,Hv,dk,dv] fp32.  o [B,N,Hv,dv]
    (q's dtype) and U [B,Hv,N,dv] fp32 are allocated when not given.
    dev_status, if given, is an int32 [B] CUDA tensor filled per sequence.
    """
    return _verify("gdn_tree_verify", q, k, v, log_alpha, beta, parent, S0, o, U, dev_status,
                   stream)


def verify_recurrent(q, k, v, log_alpha, beta, parent, S0, *, o=None, U=None, dev_status=None,
                     stream=None):
    """Single-branch recurrent verification (C ABI gdn_tree_verify_recurrent), the
    baseline the tree verification is measured against: same arguments and
    outputs as ``verify``.  Returns (o, U)."""
    return _verify("gdn_tree_verify_recurrent", q, k, v, log_alpha, beta, parent, S0, o, U,
                   dev_status, stream)


def _verify(symbol, q, k, v, log_alpha, beta, parent, S0, o, U, dev_status, stream):
    if stream is not None:
        return _on(stream, _verify, locals())
    B, N, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = q.dtype
    _check(q, "q", dt)
    _check(k, "k", dt, (B, N, Hqk, dk))
    _check(v, "v", dt, (B, N, Hv, dv))
    _check(log_alpha, "log_alpha", torch.float32, (B, N, Hv))
    _check(beta, "beta", torch.float32, (B, N, Hv))
    _check(parent, "parent", torch.int32, (B, N))
    _check(S0, "S0", torch.float32, (B, Hv, dk, dv))
    if o is None:
        o = torch.empty((B, N, Hv, dv), dtype=dt, device=q.device)
    if U is None:
        U = torch.empty((B, Hv, N, dv), dtype=torch.float32, device=q.device)
    _check(o, "o", dt, (B, N, Hv, dv))
    _check(U, "U", torch.float32, (B, Hv, N, dv))
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (B,))
    rc = getattr(load(), symbol)(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                 _ptr(parent), _ptr(S0), _ptr(o), _ptr(U), dims_of(q, v),
                                 _ptr(dev_status), _stream())
    if rc != OK:
        raise GdnTreeError(rc, symbol)
    return o, U


def commit(path, path_len, U, k, log_alpha, S0, *, S1=None, parent=None, dev_status=None,
           stream=None, dv: int | None = None):
    """Delayed state commitment (C ABI gdn_tree_commit).  Returns S1.

    path [B,Lmax] int32 (-1 padded), path_len [B] int32, U [B,Hv,N,dv] fp32
    from verify, k [B,N,Hqk,dk], log_alpha [B,N,Hv], S0 [B,Hv,dk,dv].  S1 is
    allocated when not given; pass S1=S0 for an in-place commit.  parent
    (optional) enables the chain check of the path.
    """
    if stream is not None:
        return _on(stream, commit, locals())
    B, N, Hqk, dk = k.shape
    Hv, dv = S0.shape[1], S0.shape[3]
    _check(path, "path", torch.int32)
    Lmax = path.shape[1]
    _check(path_len, "path_len", torch.int32, (B,))
    _check(U, "U", torch.float32, (B, Hv, N, dv))
    _check(k, "k")
    _check(log_alpha, "log_alpha", torch.float32, (B, N, Hv))
    _check(S0, "S0", torch.float32, (B, Hv, dk, dv))
    if S1 is None:
        S1 = torch.empty_like(S0)
    _check(S1, "S1", torch.float32, (B, Hv, dk, dv))
    if parent is not None:
        _check(parent, "parent", torch.int32, (B, N))
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (B,))
    d = Dims(B, N, Hqk, Hv, dk, dv, _dtype_code(k))
    rc = load().gdn_tree_commit(_ptr(path), _ptr(path_len), _ptr(parent), _ptr(U), _ptr(k),
                                _ptr(log_alpha), _ptr(S0), _ptr(S1), d, Lmax,
                                _ptr(dev_status), _stream())
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_commit")
    return S1


def commit_verify(prev_path, prev_path_len, prev_U, prev_k, prev_log_alpha, S_prev, q, k, v,
                  log_alpha, beta, parent, *, S1=None, prev_parent=None, o=None, U=None,
                  commit_status=None, verify_status=None, stream=None):
    """One decoding iteration (C ABI gdn_tree_commit_verify): commit the previous
    tree's accepted path into S1, then verify the next tree from S1.
    Returns (S1, o, U).  S1=S_prev commits in place; U=prev_U reuses the buffer."""
    if stream is not None:
        return _on(stream, commit_verify, locals())
    B, N, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = q.dtype
    Np = prev_k.shape[1]
    _check(prev_path, "prev_path", torch.int32)
    Lmax = prev_path.shape[1]
    _check(prev_path_len, "prev_path_len", torch.int32, (B,))
    _check(prev_U, "prev_U", torch.float32, (B, Hv, Np, dv))
    _check(prev_k, "prev_k", dt, (B, Np, Hqk, dk))
    _check(prev_log_alpha, "prev_log_alpha", torch.float32, (B, Np, Hv))
    _check(S_prev, "S_prev", torch.float32, (B, Hv, dk, dv))
    _check(q, "q", dt)
    _check(k, "k", dt, (B, N, Hqk, dk))
    _check(v, "v", dt, (B, N, Hv, dv))
    _check(log_alpha, "log_alpha", torch.float32, (B, N, Hv))
    _check(beta, "beta", torch.float32, (B, N, Hv))
    _check(parent, "parent", torch.int32, (B, N))
    if S1 is None:
        S1 = torch.empty_like(S_prev)
    if o is None:
        o = torch.empty((B, N, Hv, dv), dtype=dt, device=q.device)
    if U is None:
        U = torch.empty((B, Hv, N, dv), dtype=torch.float32, device=q.device)
    _check(S1, "S1", torch.float32, (B, Hv, dk, dv))
    _check(o, "o", dt, (B, N, Hv, dv))
    _check(U, "U", torch.float32, (B, Hv, N, dv))
    if prev_parent is not None:
        _check(prev_parent, "prev_parent", torch.int32, (B, Np))
    for name, st in (("commit_status", commit_status), ("verify_status", verify_status)):
        if st is not None:
            _check(st, name, torch.int32, (B,))
    rc = load().gdn_tree_commit_verify(
        _ptr(prev_path), _ptr(prev_path_len), _ptr(prev_parent), _ptr(prev_U), _ptr(prev_k),
        _ptr(prev_log_alpha), Np, Lmax, _ptr(S_prev), _ptr(S1), _ptr(q), _ptr(k), _ptr(v),
        _ptr(log_alpha), _ptr(beta), _ptr(parent), _ptr(o), _ptr(U), dims_of(q, v),
        _ptr(commit_status), _ptr(verify_status), _stream())
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_commit_verify")
    return S1, o, U


# ---------------------------------------------------------------------------
# packed (ragged) batches with a state pool
# ---------------------------------------------------------------------------

def _packed_rows(cu_nodes, B):
    _check(cu_nodes, "cu_nodes", torch.int32, (B + 1,))


def _slots(state_slot, B, pool):
    if state_slot is not None:
        _check(state_slot, "state_slot", torch.int32, (B,))
    return pool.shape[0]


def verify_packed(q, k, v, log_alpha, beta, parent, cu_nodes, state_pool, *, state_slot=None,
                  N_max=None, o=None, U=None, dev_status=None, stream=None):
    """Tree verification of a packed (ragged) batch (C ABI gdn_tree_verify_packed).
    Returns (o, U).

    q, k [T,Hqk,dk], v [T,Hv,dv] (bf16 or fp32); log_alpha, beta [T,Hv]; parent
    [T] (indices within each sequence); cu_nodes [B+1] int32 row offsets;
    state_pool [n_slots,Hv,dk,dv] fp32 with state_slot [B] (None: slot b).
    N_max is the largest tree (computed from cu_nodes on the host if None).
    o [T,Hv,dv] and U [Hv,T,dv] are allocated when not given."""
    if stream is not None:
        return _on(stream, verify_packed, locals())
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    B = cu_nodes.shape[0] - 1
    dt = q.dtype
    _packed_rows(cu_nodes, B)
    _check(q, "q", dt)
    _check(k, "k", dt, (T, Hqk, dk))
    _check(v, "v", dt, (T, Hv, dv))
    _check(log_alpha, "log_alpha", torch.float32, (T, Hv))
    _check(beta, "beta", torch.float32, (T, Hv))
    _check(parent, "parent", torch.int32, (T,))
    _check(state_pool, "state_pool", torch.float32, (state_pool.shape[0], Hv, dk, dv))
    n_slots = _slots(state_slot, B, state_pool)
    if N_max is None:
        N_max = int((cu_nodes[1:] - cu_nodes[:-1]).max().item()) if B > 0 else 0
    if o is None:
        o = torch.empty((T, Hv, dv), dtype=dt, device=q.device)
    if U is None:
        U = torch.empty((Hv, T, dv), dtype=torch.float32, device=q.device)
    _check(o, "o", dt, (T, Hv, dv))
    _check(U, "U", torch.float32, (Hv, T, dv))
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (B,))
    d = Dims(B, N_max, Hqk, Hv, dk, dv, _dtype_code(q))
    rc = load().gdn_tree_verify_packed(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                       _ptr(parent), _ptr(cu_nodes), T, _ptr(state_pool),
                                       _ptr(state_slot), n_slots, _ptr(o), _ptr(U), d,
                                       _ptr(dev_status), _stream())
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_verify_packed")
    return o, U


def commit_packed(path, path_len, U, k, log_alpha, cu_nodes, pool_in, *, pool_out=None,
                  state_slot=None, parent=None, N_max=None, dev_status=None, stream=None):
    """Delayed commitment of a packed batch (C ABI gdn_tree_commit_packed):
    pool_out[state_slot[b]] = the state after sequence b's accepted path.  Returns
    pool_out (pool_out=pool_in commits in place; a new pool starts as a copy of
    pool_in, so that untouched slots keep their states)."""
    if stream is not None:
        return _on(stream, commit_packed, locals())
    T, Hqk, dk = k.shape
    Hv, dv = pool_in.shape[1], pool_in.shape[3]
    B = cu_nodes.shape[0] - 1
    _packed_rows(cu_nodes, B)
    _check(path, "path", torch.int32)
    Lmax = path.shape[1]
    _check(path_len, "path_len", torch.int32, (B,))
    _check(U, "U", torch.float32, (Hv, T, dv))
    _check(k, "k")
    _check(log_alpha, "log_alpha", torch.float32, (T, Hv))
    _check(pool_in, "pool_in", torch.float32)
    n_slots = _slots(state_slot, B, pool_in)
    if pool_out is None:
        pool_out = pool_in.clone()
    _check(pool_out, "pool_out", torch.float32, tuple(pool_in.shape))
    if parent is not None:
        _check(parent, "parent", torch.int32, (T,))
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (B,))
    if N_max is None:
        N_max = int((cu_nodes[1:] - cu_nodes[:-1]).max().item()) if B > 0 else 0
    d = Dims(B, N_max, Hqk, Hv, dk, dv, _dtype_code(k))
    rc = load().gdn_tree_commit_packed(_ptr(path), _ptr(path_len), _ptr(parent), _ptr(cu_nodes),
                                       T, _ptr(U), _ptr(k), _ptr(log_alpha), _ptr(pool_in),
                                       _ptr(pool_out), _ptr(state_slot), n_slots, d, Lmax,
                                       _ptr(dev_status), _stream())
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_commit_packed")
    return pool_out


def commit_verify_packed(prev_path, prev_path_len, prev_U, prev_k, prev_log_alpha, prev_cu_nodes,
                         pool_in, q, k, v, log_alpha, beta, parent, cu_nodes, *, pool_out=None,
                         state_slot=None, prev_parent=None, prev_N_max=None, N_max=None, o=None,
                         U=None, commit_status=None, verify_status=None, stream=None):
    """One decoding iteration of a packed batch (C ABI gdn_tree_commit_verify_packed).
    Returns (pool_out, o, U); pool_out=pool_in commits in place."""
    if stream is not None:
        return _on(stream, commit_verify_packed, locals())
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    Tp = prev_k.shape[0]
    B = cu_nodes.shape[0] - 1
    dt = q.dtype
    _packed_rows(cu_nodes, B)
    _packed_rows(prev_cu_nodes, B)
    _check(prev_path, "prev_path", torch.int32)
    Lmax = prev_path.shape[1]
    _check(prev_path_len, "prev_path_len", torch.int32, (B,))
    _check(prev_U, "prev_U", torch.float32, (Hv, Tp, dv))
    _check(prev_k, "prev_k", dt, (Tp, Hqk, dk))
    _check(prev_log_alpha, "prev_log_alpha", torch.float32, (Tp, Hv))
    _check(pool_in, "pool_in", torch.float32)
    n_slots = _slots(state_slot, B, pool_in)
    _check(q, "q", dt)
    _check(k, "k", dt, (T, Hqk, dk))
    _check(v, "v", dt, (T, Hv, dv))
    _check(log_alpha, "log_alpha", torch.float32, (T, Hv))
    _check(beta, "beta", torch.float32, (T, Hv))
    _check(parent, "parent", torch.int32, (T,))
    if pool_out is None:
        pool_out = pool_in.clone()
    if o is None:
        o = torch.empty((T, Hv, dv), dtype=dt, device=q.device)
    if U is None:
        U = torch.empty((Hv, T, dv), dtype=torch.float32, device=q.device)
    _check(pool_out, "pool_out", torch.float32, tuple(pool_in.shape))
    _check(o, "o", dt, (T, Hv, dv))
    _check(U, "U", torch.float32, (Hv, T, dv))
    if prev_parent is not None:
        _check(prev_parent, "prev_parent", torch.int32, (Tp,))
    for name, st in (("commit_status", commit_status), ("verify_status", verify_status)):
        if st is not None:
            _check(st, name, torch.int32, (B,))
    if N_max is None:
        N_max = int((cu_nodes[1:] - cu_nodes[:-1]).max().item()) if B > 0 else 0
    if prev_N_max is None:
        prev_N_max = int((prev_cu_nodes[1:] - prev_cu_nodes[:-1]).max().item()) if B > 0 else 0
    d = Dims(B, N_max, Hqk, Hv, dk, dv, _dtype_code(q))
    rc = load().gdn_tree_commit_verify_packed(
        _ptr(prev_path), _ptr(prev_path_len), _ptr(prev_parent), _ptr(prev_cu_nodes), Tp,
        _ptr(prev_U), _ptr(prev_k), _ptr(prev_log_alpha), prev_N_max, Lmax, _ptr(pool_in),
        _ptr(pool_out), _ptr(state_slot), n_slots, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
        _ptr(beta), _ptr(parent), _ptr(cu_nodes), T, _ptr(o), _ptr(U), d, _ptr(commit_status),
        _ptr(verify_status), _stream())
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_commit_verify_packed")
    return pool_out, o, U


# ---------------------------------------------------------------------------
# draft-tree construction
# ---------------------------------------------------------------------------

def build_topw(cand_logp, w: int, max_depth: int, *, parent=None, cand_index=None, score=None,
               n_built=None, stream=None):
    """Top-w best-first draft-tree construction (C ABI gdn_tree_build_topw).

    cand_logp [B, N, c] fp32: the log-probabilities of each node's c candidate
    children.  Returns (parent [B, N] int32, cand_index [B, N] int32, score [B, N]
    fp32, n_built [B] int32); outputs are allocated when not given."""
    if stream is not None:
        return _on(stream, build_topw, locals())
    _check(cand_logp, "cand_logp", torch.float32)
    B, N, c = cand_logp.shape
    dev = cand_logp.device
    if parent is None:
        parent = torch.empty((B, N), dtype=torch.int32, device=dev)
    if cand_index is None:
        cand_index = torch.empty((B, N), dtype=torch.int32, device=dev)
    if score is None:
        score = torch.empty((B, N), dtype=torch.float32, device=dev)
    if n_built is None:
        n_built = torch.empty((B,), dtype=torch.int32, device=dev)
    _check(parent, "parent", torch.int32, (B, N))
    _check(cand_index, "cand_index", torch.int32, (B, N))
    _check(score, "score", torch.float32, (B, N))
    _check(n_built, "n_built", torch.int32, (B,))
    rc = load().gdn_tree_build_topw(_ptr(cand_logp), B, N, c, w, max_depth, _ptr(parent),
                                    _ptr(cand_index), _ptr(score), _ptr(n_built),
                                    _stream())
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_build_topw")
    return parent, cand_index, score, n_built


# ---------------------------------------------------------------------------
# serving a hybrid model: prefill, decoding step, attention, cache
# ---------------------------------------------------------------------------

def _most_rows(cu) -> int:
    return int((cu[1:] - cu[:-1]).max().item()) if cu.shape[0] > 1 else 0


def _workspace(given, need, device):
    """The workspace to pass: the caller's, one of our own, or none where none is needed."""
    if given is not None:
        _check(given, "workspace", torch.uint8)
        if given.numel() < need:
            raise ValueError(f"workspace has {given.numel()} bytes, {need} are needed")
    return None if not need else given if given is not None else torch.empty(
        need, dtype=torch.uint8, device=device)


_struct_cache: dict = {}


def _struct(kind, *key):
    """kind(*key), kept by its values to save the rebuild."""
    d = _struct_cache.get((kind, key))
    if d is None:
        d = kind(*key)
        if len(_struct_cache) < 256:
            _struct_cache[kind, key] = d
    return d


_prefill_cache: dict = {}


def prefill_workspace(dims: Dims, T: int) -> int:
    """Bytes of device memory that ``prefill`` needs for these dims and T rows."""
    return load().gdn_tree_prefill_workspace(dims, T)


def prefill(q, k, v, log_alpha, beta, cu_tokens, state_pool, *, state_slot=None, N_max=None,
            pool_out=None, o=None, workspace=None, dev_status=None, stream=None):
    """The gated delta rule over whole sequences (C ABI gdn_tree_prefill).
    Returns (o, pool_out).

    q, k [T,Hqk,dk], v [T,Hv,dv] (bf16 or fp32); log_alpha, beta [T,Hv]; cu_tokens [B+1]
    int32 row offsets; state_pool [n_slots,Hv,dk,dv] fp32 with state_slot [B] (None: slot
    b) holds the state each sequence starts from.  o [T,Hv,dv] is allocated when not given;
    pool_out=state_pool updates in place, a new pool starts as a copy of state_pool.
    workspace (``prefill_workspace`` bytes, uint8) is allocated when not given.  N_max is the longest sequence (computed from cu_tokens on the host if None)."""
    if stream is not None:
        return _on(stream, prefill, locals())
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    B = cu_tokens.shape[0] - 1
    dt = q.dtype
    code = _dtype_code(q)
    _check(cu_tokens, "cu_tokens", torch.int32, (B + 1,))
    _check(q, "q", dt)
    _check(k, "k", dt, (T, Hqk, dk))
    _check(v, "v", dt, (T, Hv, dv))
    _check(log_alpha, "log_alpha", torch.float32, (T, Hv))
    _check(beta, "beta", torch.float32, (T, Hv))
    _check(state_pool, "state_pool", torch.float32, (state_pool.shape[0], Hv, dk, dv))
    n_slots = _slots(state_slot, B, state_pool)
    if N_max is None:
        N_max = _most_rows(cu_tokens)
    if pool_out is None:
        pool_out = state_pool.clone()
    if o is None:
        o = torch.empty((T, Hv, dv), dtype=dt, device=q.device)
    _check(pool_out, "pool_out", torch.float32, state_pool.shape)
    _check(o, "o", dt, (T, Hv, dv))
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (B,))
    key = (B, N_max, Hqk, Hv, dk, dv, code, T)
    known = _prefill_cache.get(key)
    if known is None:
        d = Dims(*key[:7])
        known = d, prefill_workspace(d, T)
        if len(_prefill_cache) < 256:
            _prefill_cache[key] = known
    d, need = known
    workspace = _workspace(workspace, need, q.device)
    rc = load().gdn_tree_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                 _ptr(cu_tokens), T, _ptr(state_pool), _ptr(pool_out),
                                 _ptr(state_slot), n_slots, _ptr(o), d, _ptr(dev_status),
                                 _ptr(workspace), need, _stream())
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_prefill")
    return o, pool_out


def decode_step(q, k, v, log_alpha, beta, state_pool, *, state_slot=None, pool_out=None, o=None,
                dev_status=None, stream=None):
    """The gated delta rule for one token of each sequence (C ABI gdn_tree_decode_step).
    Returns (o, pool_out).

    q, k [B,Hqk,dk], v [B,Hv,dv] (bf16 or fp32); log_alpha, beta [B,Hv] fp32; state_pool
    [n_slots,Hv,dk,dv] fp32 with state_slot [B] (None: slot b).  pool_out=state_pool steps
    in place; a new pool starts as a copy of state_pool."""
    if stream is not None:
        return _on(stream, decode_step, locals())
    B, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    dt = q.dtype
    code = _dtype_code(q)
    _check(q, "q", dt)
    _check(k, "k", dt, (B, Hqk, dk))
    _check(v, "v", dt, (B, Hv, dv))
    _check(log_alpha, "log_alpha", torch.float32, (B, Hv))
    _check(beta, "beta", torch.float32, (B, Hv))
    _check(state_pool, "state_pool", torch.float32, (state_pool.shape[0], Hv, dk, dv))
    n_slots = _slots(state_slot, B, state_pool)
    if pool_out is None:
        pool_out = state_pool.clone()
    if o is None:
        o = torch.empty((B, Hv, dv), dtype=dt, device=q.device)
    _check(pool_out, "pool_out", torch.float32, state_pool.shape)
    _check(o, "o", dt, (B, Hv, dv))
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (B,))
    rc = load().gdn_tree_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                     _ptr(state_pool), _ptr(pool_out), _ptr(state_slot), n_slots,
                                     _ptr(o), _struct(Dims, B, 1, Hqk, Hv, dk, dv, code),
                                     _ptr(dev_status), _stream())
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_decode_step")
    return o, pool_out


def _check_cache(k_cache, v_cache, page_table, context_len, B, Hkv, D, dt):
    n_pages, page = k_cache.shape[0], k_cache.shape[1]
    _check(k_cache, "k_cache", dt, (n_pages, page, Hkv, D))
    _check(v_cache, "v_cache", dt, (n_pages, page, Hkv, D))
    _check(page_table, "page_table", torch.int32, (B, page_table.shape[1]))
    _check(context_len, "context_len", torch.int32, (B,))
    return n_pages, page, page_table.shape[1]


def attend_workspace(dims: AttendDims) -> int:
    """Bytes of device memory that ``attend`` needs for these dims."""
    return load().gdn_tree_attend_workspace(dims)


_attend_cache: dict = {}


def attend(q, k, v, parent, cu_nodes, k_cache, v_cache, page_table, context_len, *,
           prefix_pages=None, prefix_len=0, scale=None, N_max=None, o=None, lse=None,
           workspace=None, dev_status=None, stream=None):
    """Attention of draft trees over a paged cache with a shared prefix (C ABI
    gdn_tree_attend).  Returns (o, lse).

    q [T,Hq,D] and the rows' own k, v [T,Hkv,D] (both None: the rows see the cache alone);
    parent [T] int32, trees of up to 1024 rows (None: every sequence's rows are a chain of
    any length, causal attention); cu_nodes
    [B+1]; k_cache, v_cache [n_pages,page_size,Hkv,D]; page_table [B,width] int32 and
    context_len [B] int32: each sequence's own context; prefix_pages [ceil(prefix_len /
    page_size)] int32: the rows that every sequence sees before its own.  scale defaults to
    1/sqrt(D).  o [T,Hq,D], lse [T,Hq] fp32 and workspace (``attend_workspace`` bytes, uint8)
    are allocated when not given.  N_max is the most rows of one sequence (computed from
    cu_nodes on the host if None)."""
    if stream is not None:
        return _on(stream, attend, locals())
    T, Hq, D = q.shape
    B = cu_nodes.shape[0] - 1
    Hkv = k_cache.shape[2]
    dt = q.dtype
    code = _dtype_code(q)
    _check(q, "q", dt)
    if (k is None) != (v is None):
        raise ValueError("k and v are given together or not at all")
    if k is not None:
        _check(k, "k", dt, (T, Hkv, D))
        _check(v, "v", dt, (T, Hkv, D))
    if parent is not None:
        _check(parent, "parent", torch.int32, (T,))
    _check(cu_nodes, "cu_nodes", torch.int32, (B + 1,))
    n_pages, page, width = _check_cache(k_cache, v_cache, page_table, context_len, B, Hkv, D, dt)
    if prefix_len:
        _check(prefix_pages, "prefix_pages", torch.int32, (-(-prefix_len // page),))
    if N_max is None:
        N_max = _most_rows(cu_nodes)
    if o is None:
        o = torch.empty((T, Hq, D), dtype=dt, device=q.device)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    _check(o, "o", dt, (T, Hq, D))
    _check(lse, "lse", torch.float32, (T, Hq))
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (B,))
    lib = load()
    key = (B, T, N_max, Hq, Hkv, D, code, page, n_pages, width, prefix_len)
    known = _attend_cache.get(key)
    if known is None:
        d = AttendDims(*key)
        known = d, lib.gdn_tree_attend_workspace(d)
        if len(_attend_cache) < 256:
            _attend_cache[key] = known
    d, need = known
    workspace = _workspace(workspace, need, q.device)
    rc = lib.gdn_tree_attend(_ptr(q), _ptr(k), _ptr(v), _ptr(parent), _ptr(cu_nodes),
                             _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(context_len),
                             _ptr(prefix_pages) if prefix_len else None,
                             D ** -0.5 if scale is None else scale, _ptr(o), _ptr(lse), d,
                             _ptr(dev_status), _ptr(workspace), need,
                             _stream())
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_attend")
    return o, lse


def cache_append(k, v, cu_nodes, k_cache, v_cache, page_table, context_len, *, path=None,
                 path_len=None, N_max=None, new_len=None, dev_status=None, stream=None):
    """Rows join the paged cache of their sequences (C ABI gdn_tree_cache_append): the
    attention's counterpart of ``commit``.  Returns new_len [B] int32, the context lengths
    after the call.

    k, v [T,Hkv,D]; with path [B,Lmax] and path_len [B] int32 the accepted nodes of each
    tree, else all rows of each sequence.  k_cache, v_cache [n_pages,page_size,Hkv,D] are
    written in place at rows context_len[b] .. of the pages that page_table [B,width]
    already holds.  context_len itself is not changed."""
    if stream is not None:
        return _on(stream, cache_append, locals())
    T, Hkv, D = k.shape
    B = cu_nodes.shape[0] - 1
    dt = k.dtype
    code = _dtype_code(k)
    _check(k, "k", dt)
    _check(v, "v", dt, (T, Hkv, D))
    _check(cu_nodes, "cu_nodes", torch.int32, (B + 1,))
    n_pages, page, width = _check_cache(k_cache, v_cache, page_table, context_len, B, Hkv, D, dt)
    Lmax = 0
    if (path is None) != (path_len is None):
        raise ValueError("path and path_len are given together or not at all")
    if path is not None:
        Lmax = path.shape[1]
        _check(path, "path", torch.int32, (B, Lmax))
        _check(path_len, "path_len", torch.int32, (B,))
    if N_max is None:
        N_max = _most_rows(cu_nodes)
    if new_len is None:
        new_len = torch.empty((B,), dtype=torch.int32, device=k.device)
    _check(new_len, "new_len", torch.int32, (B,))
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (B,))
    d = _struct(AttendDims, B, T, N_max, Hkv, Hkv, D, code, page, n_pages, width, 0)
    rc = load().gdn_tree_cache_append(_ptr(k), _ptr(v), _ptr(path), _ptr(path_len), Lmax,
                                      _ptr(cu_nodes), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(page_table), _ptr(context_len), _ptr(new_len), d,
                                      _ptr(dev_status), _stream())
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_cache_append")
    return new_len


# ---------------------------------------------------------------------------
# in front of the attention: positions, norms and rotation
# ---------------------------------------------------------------------------

# (These take 4 to 18 tensors ahead of a launch of 2 microseconds.  So that a call costs little
# where nothing is wrong, its tensors are looked at in one expression, each property read once;
# where that finds a fault, or what it does not know, they are checked one by one, which says what
# is wrong.  What the call needs of the shapes is made once for each set of them.)

_i32, _i64, _f32 = torch.int32, torch.int64, torch.float32
_CODES = {torch.bfloat16: BF16, torch.float32: F32}
# (asked only where there is a CUDA tensor: the runtime is up then)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(dev) -> int:
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _check_device(t, name, dev):
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device than the current one")


def _check_flat(dev, *tensors):
    """Dense tensors (tensor or None, name, type, shape) on the current device."""
    for t, name, dtype, shape in tensors:
        if t is not None:
            _check(t, name, dtype, shape)
            _check_device(t, name, dev)


def _check_heads(dev, dtype, T, D, *tensors):
    """Arrays of heads [T,H,D] (tensor or None, name, the tensor whose shape it has or None) whose
    heads are contiguous."""
    for t, name, like in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        H = t.shape[1] if like is None and t.dim() > 1 else "H" if like is None else like.shape[1]
        if t.shape != (T, H, D):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(T, H, D)}")
        if t.stride(2) != 1 and t.numel():
            raise ValueError(f"{name}'s heads must be contiguous")
        _check_device(t, name, dev)


def _refuse_device(t, name):
    """Refuses t, which is not on the current device."""
    raise ValueError(f"{name} must be a CUDA tensor" if t.get_device() < 0 else
                     f"{name} is on another device than the current one")


_LOW, _HIGH = -(1 << 31), (1 << 31) - 1


def _check_int32(**values):
    """Refuses what a 32-bit argument does not hold (ctypes would wrap it without a word)."""
    for name, x in values.items():
        if not _LOW <= x <= _HIGH:
            raise ValueError(f"{name} is {x}, which 32 bits do not hold")


_NO_STRIDES = (0, 0, 0)
_DIMS = ("B", "T", "N_max", "Hq", "Hkv", "D", "dtype", "page_size", "n_pages", "table_width",
         "prefix_len")
_rope_cache: dict = {}


def _rope_structs(strides, dims, interleaved, norm, rope_scale, eps, R):
    """The structs of a call, HeadStrides, AttendDims and Rope, kept by their values (which are
    plain numbers here: a tensor would be known by its identity)."""
    interleaved = bool(interleaved)
    key = (strides, dims, interleaved, norm, rope_scale, eps, R)
    known = _rope_cache.get(key)
    if known is None:
        if norm not in NORMS:
            raise ValueError(f"norm must be one of {list(NORMS)}, got {norm!r}")
        _check_int32(rotary_dim=R, **dict(zip(_DIMS, dims)))
        known = (HeadStrides(*(Strides(*s[:2]) for s in strides)), AttendDims(*dims),
                 Rope(R, interleaved, NORMS[norm], rope_scale, eps))
        if len(_rope_cache) >= 256:  # (a server's rows differ from call to call)
            _rope_cache.clear()
        _rope_cache[key] = known
    return known


def tree_positions(parent, cu_nodes, *, context_len=None, prefix_len=0, T=None, N_max=None,
                   positions=None, dev_status=None, stream=None):
    """The positions of draft trees' nodes, or of chains' rows (C ABI gdn_tree_positions):
    prefix_len + context_len[b] + the node's depth.  Returns positions [T] int32.

    parent [T] int32, trees of up to 1024 rows (None: every sequence's rows are a chain of any
    length; T or positions then says how many rows there are); cu_nodes [B+1]; context_len [B]
    int32 (None: 0).  positions is allocated when not given; rows of no sequence are left as
    they are (of an allocated one: anything)."""
    if stream is not None:
        return _on(stream, tree_positions, locals())
    dev = cu_nodes.get_device()
    if dev < 0 or dev != _current_device():
        _refuse_device(cu_nodes, "cu_nodes")
    B = cu_nodes.shape[0] - 1
    if parent is not None:
        rows = parent.shape[0]
    elif positions is not None:
        rows = positions.shape[0]
    elif T is not None:
        rows = T
    else:
        raise ValueError("without parent, T or positions says how many rows there are")
    if T is not None and T != rows:
        raise ValueError(f"T is {T}, but there are {rows} rows")
    if positions is None:
        positions = torch.empty((rows,), dtype=torch.int32, device=cu_nodes.device)
    try:
        good = (cu_nodes.dtype is _i32 and cu_nodes.is_contiguous() and cu_nodes.dim() == 1
                and positions.shape == (rows,) and positions.dtype is _i32
                and positions.is_contiguous() and positions.get_device() == dev
                and (parent is None or parent.dtype is _i32 and parent.is_contiguous()
                     and parent.dim() == 1 and parent.get_device() == dev)
                and (context_len is None or context_len.shape == (B,) and context_len.dtype is _i32
                     and context_len.is_contiguous() and context_len.get_device() == dev)
                and (dev_status is None or dev_status.shape == (B,) and dev_status.dtype is _i32
                     and dev_status.is_contiguous() and dev_status.get_device() == dev))
    except AttributeError:  # (no tensor)
        good = False
    if not good:
        _check_flat(dev, (cu_nodes, "cu_nodes", torch.int32, (B + 1,)),
                    (parent, "parent", torch.int32, (rows,)),
                    (context_len, "context_len", torch.int32, (B,)),
                    (positions, "positions", torch.int32, (rows,)),
                    (dev_status, "dev_status", torch.int32, (B,)))
    if N_max is None:
        N_max = _most_rows(cu_nodes)
    prefix_len, N_max = index(prefix_len), index(N_max)
    if not (_LOW <= prefix_len <= _HIGH and _LOW <= N_max <= _HIGH and B <= _HIGH
            and rows <= _HIGH):
        _check_int32(prefix_len=prefix_len, N_max=N_max, B=B, T=rows)
    rc = load().gdn_tree_positions(
        None if parent is None else parent.data_ptr(), cu_nodes.data_ptr(),
        None if context_len is None else context_len.data_ptr(), prefix_len,
        positions.data_ptr(), B, rows, N_max,
        None if dev_status is None else dev_status.data_ptr(), _stream_of(dev))
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_positions")
    return positions


def rope_frequencies(rotary_dim, base=10000.0, *, stretch=None, factor=1.0, trained_len=0.0,
                     fast=32.0, slow=1.0, device="cuda"):
    """A model's rotary frequencies (C ABI gdn_tree_rope_frequencies), made once.  Returns
    (freq [rotary_dim / 2] int64, rope_scale), as ``norm_rope`` takes them: freq is turns a
    position in units of 2^-64.

    stretch, for positions past those of the training: None, "linear" (slower by factor), "ntk"
    (a larger base), "yarn" or "bands" (pairs that turn `slow` times or less in trained_len
    positions are slower by factor, those that turn `fast` times or more keep their speed)."""
    if stretch not in STRETCHES:
        raise ValueError(f"stretch must be one of {list(STRETCHES)}, got {stretch!r}")
    _check_int32(rotary_dim=rotary_dim)
    # (more than the library takes are refused before they are written)
    freq = (ctypes.c_uint64 * min(max(int(rotary_dim) // 2, 1), 1 << 16))()
    scale = ctypes.c_float()
    rc = load().gdn_tree_rope_frequencies(
        rotary_dim, base, RopeStretch(STRETCHES[stretch], factor, trained_len, fast, slow), freq,
        ctypes.byref(scale))
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_rope_frequencies")
    # (all below 2^63)
    return torch.tensor(list(freq), dtype=torch.int64, device=device), scale.value


def norm_rope(q, k=None, positions=None, freq=None, *, interleaved=False, rope_scale=1.0,
              norm=None, q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None,
              stream=None):
    """Queries and keys normalised for each head and rotated by their rows' positions, in one
    pass (C ABI gdn_tree_norm_rope).  Returns (q_out, k_out), None for one that is not given.

    q [T,Hq,D], k [T,Hkv,D] (bf16 or fp32; either may be None), heads contiguous, rows and heads
    with any strides of whole 16 bytes: columns of a projection's output need no copy.  norm:
    None, "rms" (with q_weight, k_weight [D] fp32, or without) or "unit".  positions [T] int32
    and freq [R/2] (``rope_frequencies``) rotate the first R elements of each head, element i
    with i + R/2 or, interleaved, 2 i with 2 i + 1; both None: no rotation.  q_out, k_out are
    allocated when not given; q_out=q and k_out=k work in place."""
    if stream is not None:
        return _on(stream, norm_rope, locals())
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k must be given")
    if (positions is None) != (freq is None):
        raise ValueError("positions and freq are given together or not at all")
    T, _, D = x.shape
    dt = x.dtype
    code = _CODES.get(dt)
    if code is None:
        _dtype_code(x)
    dev = x.get_device()
    if dev < 0 or dev != _current_device():
        _refuse_device(x, "q" if x is q else "k")
    Hq = Hkv = R = 0
    qs = ks = qo = ko = _NO_STRIDES
    qp = kp = qop = kop = pp = fp = wq = wk = None
    q_shape = k_shape = f_shape = None
    good = True
    try:
        if q is not None:
            q_shape = q.shape
            if q_out is None:
                q_out = torch.empty(q_shape, dtype=dt, device=q.device)
            Hq, qs, qo = q_shape[1], q.stride(), q_out.stride()
            good = (qs[2] == 1 and qo[2] == 1 and q_out.shape == q_shape and q_out.dtype is dt
                    and q_out.get_device() == dev
                    and (q_weight is None or q_weight.shape == (D,) and q_weight.dtype is _f32
                         and q_weight.is_contiguous() and q_weight.get_device() == dev))
            qp, qop = q.data_ptr(), q_out.data_ptr()
            wq = None if q_weight is None else q_weight.data_ptr()
        elif q_out is not None:
            raise ValueError("q_out is given with q")
        if k is not None:
            k_shape = k.shape
            if k_out is None:
                k_out = torch.empty(k_shape, dtype=dt, device=k.device)
            Hkv, ks, ko = k_shape[1], k.stride(), k_out.stride()
            good = (good and k_shape == (T, Hkv, D) and k.dtype is dt and k.get_device() == dev
                    and ks[2] == 1 and ko[2] == 1 and k_out.shape == k_shape
                    and k_out.dtype is dt and k_out.get_device() == dev
                    and (k_weight is None or k_weight.shape == (D,) and k_weight.dtype is _f32
                         and k_weight.is_contiguous() and k_weight.get_device() == dev))
            kp, kop = k.data_ptr(), k_out.data_ptr()
            wk = None if k_weight is None else k_weight.data_ptr()
        elif k_out is not None:
            raise ValueError("k_out is given with k")
        if freq is not None:
            f_shape = freq.shape
            R = 2 * f_shape[0]
            good = (good and len(f_shape) == 1 and freq.dtype is _i64 and freq.is_contiguous()
                    and freq.get_device() == dev and positions.shape == (T,)
                    and positions.dtype is _i32 and positions.is_contiguous()
                    and positions.get_device() == dev)
            fp, pp = freq.data_ptr(), positions.data_ptr()
    except (AttributeError, IndexError):  # (no tensor, or too few dimensions)
        good = False
    if not good:
        _check_heads(dev, dt, T, D, (q, "q", None), (q_out, "q_out", q), (k, "k", None),
                     (k_out, "k_out", k))
        _check_flat(dev, (q_weight if q is not None else None, "q_weight", torch.float32, (D,)),
                    (k_weight if k is not None else None, "k_weight", torch.float32, (D,)),
                    (freq, "freq", torch.int64, (R // 2,)),
                    (positions, "positions", torch.int32, (T,)))
    strides, dims, rope = _rope_structs((qs, ks, _NO_STRIDES, qo, ko),
                                        (0, T, 0, Hq, Hkv, D, code, 1, 0, 0, 0), interleaved, norm,
                                        float(rope_scale), float(eps), R)
    rc = load().gdn_tree_norm_rope(qp, kp, pp, fp, wq, wk, qop, kop, strides, dims, rope,
                                   _stream_of(dev))
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_norm_rope")
    return q_out, k_out


def cache_append_rope(q, k, v, cu_nodes, k_cache, v_cache, page_table, context_len, freq=None, *,
                      prefix_len=0, interleaved=False, rope_scale=1.0, norm=None, q_weight=None,
                      k_weight=None, eps=1e-6, q_out=None, k_out=None, v_out=None, N_max=None,
                      new_len=None, dev_status=None, stream=None):
    """All rows of each sequence join its paged cache, keys normalised and rotated on the way
    (C ABI gdn_tree_cache_append_rope).  Returns (q_out, new_len).

    Row j of sequence b stands at position prefix_len + context_len[b] + j.  k, v [T,Hkv,D] and
    q [T,Hq,D] (None: keys and values alone) with strides as for ``norm_rope``, whose freq,
    interleaved, rope_scale, norm, weights and eps these are.  k_cache, v_cache
    [n_pages,page_size,Hkv,D] are written in place, as by ``cache_append``.  q_out (the queries
    normalised and rotated) is allocated when not given, and then holds anything in the rows of no
    sequence (in a given one they are left as they are); k_out and v_out, where given, get the
    rows' keys and values too (what ``attend`` takes beside the cache).  context_len itself is
    not changed: new_len [B] int32 holds the lengths after the call."""
    if stream is not None:
        return _on(stream, cache_append_rope, locals())
    shape = k.shape
    T, Hkv, D = shape
    B = cu_nodes.shape[0] - 1
    dt = k.dtype
    code = _CODES.get(dt)
    if code is None:
        _dtype_code(k)
    dev = k.get_device()
    if dev < 0 or dev != _current_device():
        _refuse_device(k, "k")
    cache = k_cache.shape
    n_pages, page = cache[:2]
    width = page_table.shape[1]
    if new_len is None:
        new_len = torch.empty((B,), dtype=torch.int32, device=k.device)
    Hq = R = 0
    ks = vs = _NO_STRIDES
    qs = qo = ko = vo = _NO_STRIDES
    qp = qop = kop = vop = fp = wq = wk = sp = None
    try:
        ks, vs = k.stride(), v.stride()
        good = (ks[2] == 1 and vs[2] == 1 and v.shape == shape and v.dtype is dt
                and v.get_device() == dev and cu_nodes.dim() == 1 and cu_nodes.dtype is _i32
                and cu_nodes.is_contiguous() and cu_nodes.get_device() == dev
                and cache == (n_pages, page, Hkv, D) and k_cache.dtype is dt
                and k_cache.is_contiguous() and k_cache.get_device() == dev
                and v_cache.shape == cache and v_cache.dtype is dt and v_cache.is_contiguous()
                and v_cache.get_device() == dev
                and page_table.shape == (B, width) and page_table.dtype is _i32
                and page_table.is_contiguous() and page_table.get_device() == dev
                and context_len.shape == (B,) and context_len.dtype is _i32
                and context_len.is_contiguous() and context_len.get_device() == dev
                and new_len.shape == (B,) and new_len.dtype is _i32 and new_len.is_contiguous()
                and new_len.get_device() == dev)
        if q is not None:
            q_shape = q.shape
            if q_out is None:
                q_out = torch.empty(q_shape, dtype=dt, device=k.device)
            Hq, qs, qo = q_shape[1], q.stride(), q_out.stride()
            good = (good and q_shape == (T, Hq, D) and q.dtype is dt and q.get_device() == dev
                    and qs[2] == 1 and qo[2] == 1 and q_out.shape == q_shape
                    and q_out.dtype is dt and q_out.get_device() == dev
                    and (q_weight is None or q_weight.shape == (D,) and q_weight.dtype is _f32
                         and q_weight.is_contiguous() and q_weight.get_device() == dev))
            qp, qop = q.data_ptr(), q_out.data_ptr()
            wq = None if q_weight is None else q_weight.data_ptr()
        elif q_out is not None:
            raise ValueError("q_out is given with q")
        if k_out is not None:
            ko = k_out.stride()
            good = (good and ko[2] == 1 and k_out.shape == shape and k_out.dtype is dt
                    and k_out.get_device() == dev)
            kop = k_out.data_ptr()
        if v_out is not None:
            vo = v_out.stride()
            good = (good and vo[2] == 1 and v_out.shape == shape and v_out.dtype is dt
                    and v_out.get_device() == dev)
            vop = v_out.data_ptr()
        if k_weight is not None:
            good = (good and k_weight.shape == (D,) and k_weight.dtype is _f32
                    and k_weight.is_contiguous() and k_weight.get_device() == dev)
            wk = k_weight.data_ptr()
        if freq is not None:
            f_shape = freq.shape
            R = 2 * f_shape[0]
            good = (good and len(f_shape) == 1 and freq.dtype is _i64 and freq.is_contiguous()
                    and freq.get_device() == dev)
            fp = freq.data_ptr()
        if dev_status is not None:
            good = (good and dev_status.shape == (B,) and dev_status.dtype is _i32
                    and dev_status.is_contiguous() and dev_status.get_device() == dev)
            sp = dev_status.data_ptr()
    except (AttributeError, IndexError):  # (no tensor, or too few dimensions)
        good = False
    if not good:
        _check_heads(dev, dt, T, D, (q, "q", None), (q_out, "q_out", q), (k, "k", None),
                     (v, "v", k), (k_out, "k_out", k), (v_out, "v_out", k))
        _check_cache(k_cache, v_cache, page_table, context_len, B, Hkv, D, dt)
        _check_flat(dev, (cu_nodes, "cu_nodes", torch.int32, (B + 1,)),
                    (k_cache, "k_cache", dt, cache), (v_cache, "v_cache", dt, cache),
                    (page_table, "page_table", torch.int32, (B, width)),
                    (context_len, "context_len", torch.int32, (B,)),
                    (new_len, "new_len", torch.int32, (B,)),
                    (dev_status, "dev_status", torch.int32, (B,)),
                    (q_weight if q is not None else None, "q_weight", torch.float32, (D,)),
                    (k_weight, "k_weight", torch.float32, (D,)),
                    (freq, "freq", torch.int64, (R // 2,)))
    if N_max is None:
        N_max = _most_rows(cu_nodes)
    strides, dims, rope = _rope_structs(
        (qs, ks, vs, qo, ko, vo),
        (B, T, index(N_max), Hq, Hkv, D, code, page, n_pages, width, index(prefix_len)),
        interleaved, norm, float(rope_scale), float(eps), R)
    rc = load().gdn_tree_cache_append_rope(
        qp, k.data_ptr(), v.data_ptr(), fp, wq, wk, cu_nodes.data_ptr(), qop, kop, vop,
        k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), context_len.data_ptr(),
        new_len.data_ptr(), strides, dims, rope, sp, _stream_of(dev))
    if rc != OK:
        raise GdnTreeError(rc, "gdn_tree_cache_append_rope")
    return q_out, new_len
