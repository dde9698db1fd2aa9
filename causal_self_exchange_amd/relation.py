"""Thin Python binding over librelation.so (ctypes).

Argument marshalling only: every step of the forward, backward and decode runs in the
HIP kernels behind the C ABI (include/relation.h). PyTorch supplies device
memory and the current stream. There is no CPU fallback: if the library is
missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librelation.so")

REL_F32, REL_BF16, REL_E4M3 = 0, 1, 2
_DT = {torch.float32: REL_F32, torch.bfloat16: REL_BF16}

_lib = None


class RelationError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib().relation_status_str(status).decode()
        super().__init__(f"{fn} failed: status {status} ({msg})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load librelation.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run causal_self_exchange_amd.build first")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, fp, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.POINTER(ctypes.c_float), ctypes.c_size_t
        L.relation_fwd.argtypes = [vp, vp, vp, fp, vp, i, i, i, i, i, vp]
        L.relation_fwd.restype = i
        L.relation_fwd_ex.argtypes = [vp, vp, vp, fp, f, vp, i, i, i, i, i, vp]
        L.relation_fwd_ex.restype = i
        L.relation_fwd_lse.argtypes = [vp, vp, vp, fp, f, vp, vp, i, i, i, i, i, vp]
        L.relation_fwd_lse.restype = i
        L.relation_bwd_workspace_bytes.argtypes = [i, i, i, i]
        L.relation_bwd_workspace_bytes.restype = sz
        L.relation_bwd_stored_workspace_bytes.argtypes = [i, i, i, i]
        L.relation_bwd_stored_workspace_bytes.restype = sz
        L.relation_bwd.argtypes = [vp, vp, vp, fp, f, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, sz, vp]
        L.relation_bwd.restype = i
        L.relation_prestep.argtypes = [vp, vp, vp, vp, i, f, fp, i, vp, vp, vp, i, i, i, i, i, vp]
        L.relation_prestep.restype = i
        L.relation_fwd_model_workspace_bytes.argtypes = [i, i, i, i, i]
        L.relation_fwd_model_workspace_bytes.restype = sz
        L.relation_fwd_model.argtypes = [vp, vp, vp, vp, i, f, fp, i, fp, f, vp, vp, i, i, i, i, i, vp, sz, vp]
        L.relation_fwd_model.restype = i
        L.relation_linear_workspace_bytes.argtypes = [i, i, i, i]
        L.relation_linear_workspace_bytes.restype = sz
        L.relation_linear_fwd.argtypes = [vp, vp, vp, vp, fp, vp, vp, i, i, i, i, i, vp, sz, vp]
        L.relation_linear_fwd.restype = i
        L.relation_decode_workspace_bytes.argtypes = [i, i, i, i]
        L.relation_decode_workspace_bytes.restype = sz
        L.relation_decode.argtypes = [vp, vp, vp, vp, vp, vp, fp, f, vp, i, i, i, i, i, vp, sz, vp]
        L.relation_decode.restype = i
        L.relation_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, fp, f, vp, i, i, i, i, i, vp]
        L.relation_decode_noalloc.restype = i
        L.relation_cache_append.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, vp]
        L.relation_cache_append.restype = i
        l64 = ctypes.c_int64
        L.relation_page_map.argtypes = [vp] * 10 + [i] * 6 + [vp]
        L.relation_page_map.restype = i
        L.relation_paged_append.argtypes = [vp, vp, vp, l64, l64, l64, vp, vp, i, f, fp, i, vp, vp, vp,
                                            i, i, i, i, i, i, i, vp]
        L.relation_paged_append.restype = i
        L.relation_paged_workspace_bytes.argtypes = [i, i, i, i, i]
        L.relation_paged_workspace_bytes.restype = sz
        L.relation_paged_fwd.argtypes = [vp, l64, vp, vp, vp, vp, vp, fp, f, vp, i, i, i, i, i, i, i, i, i, i,
                                         vp, sz, vp]
        L.relation_paged_fwd.restype = i
        L.relation_paged_append_q8.argtypes = [vp, vp, vp, l64, l64, l64, vp, vp, i, f, ctypes.POINTER(ctypes.c_double), i,
                                               vp, vp, vp, vp, i, i, i, i, i, i, vp]
        L.relation_paged_append_q8.restype = i
        L.relation_tree_plan.argtypes = [vp] * 5 + [i] * 3 + [vp]
        L.relation_tree_plan.restype = i
        L.relation_paged_fwd_ex.argtypes = [vp, l64, vp, vp, vp, vp, vp, vp, vp, i, fp, f, vp] + [i] * 10 + [vp, sz, vp]
        L.relation_paged_fwd_ex.restype = i
        L.relation_paged_keep.argtypes = [vp] * 12 + [i] * 9 + [vp]
        L.relation_paged_keep.restype = i
        L.relation_status_str.argtypes = [i]
        L.relation_status_str.restype = ctypes.c_char_p
        L.relation_select_kernels.argtypes = [i, i]
        L.relation_select_kernels.restype = i
        _lib = L
    return _lib


EXPORTS = ("relation_fwd", "relation_fwd_ex", "relation_fwd_lse", "relation_bwd_workspace_bytes",
           "relation_bwd_stored_workspace_bytes", "relation_bwd", "relation_prestep", "relation_fwd_model_workspace_bytes",
           "relation_fwd_model", "relation_linear_workspace_bytes", "relation_linear_fwd",
           "relation_decode_workspace_bytes", "relation_decode", "relation_decode_noalloc",
           "relation_cache_append", "relation_page_map", "relation_paged_append",
           "relation_paged_workspace_bytes", "relation_paged_fwd", "relation_paged_append_q8", "relation_tree_plan",
           "relation_paged_fwd_ex", "relation_paged_keep", "relation_status_str", "relation_select_kernels")

KERNELS = {"auto": 0, "scan": 1}


def select_kernels(fwd: str = "auto", bwd: str = "auto"):
    """Process-wide choice of the bf16 forward / backward kernels: "auto"
    (the MFMA kernels wherever they apply) or "scan" (the row-scan kernels;
    paged_fwd: no query tiles, whose weights are rounded to bf16)."""
    _check("relation_select_kernels", lib().relation_select_kernels(KERNELS[fwd], KERNELS[bwd]))


class kernels:
    """Context manager: select kernels for the block, then back to "auto"."""

    def __init__(self, fwd: str = "auto", bwd: str = "auto"):
        self.sel = (fwd or "auto", bwd or "auto")

    def __enter__(self):
        select_kernels(*self.sel)
        return self

    def __exit__(self, *exc):
        select_kernels("auto", "auto")

ROPE = {"none": 0, "interleaved": 1, "half": 2}
PAIRS = {"A": 0, "B": 1}


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _tau_arg(tau, H: int):
    arr = np.ascontiguousarray(np.broadcast_to(np.asarray(tau, dtype=np.float32), (H,)))
    return arr, arr.ctypes.data_as(ctypes.POINTER(ctypes.c_float))


def _check(fn: str, st: int):
    if st != 0:
        raise RelationError(fn, st)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


class _Args:
    """Checks of caller-supplied tensors before anything reaches the library
    (which sees bare pointers and sizes and cannot check them). Every tensor
    is first checked for its shape and dtype (all of them, so a mismatch is
    reported whatever device the tensors are on), then for being a contiguous
    tensor on the device of the first one."""

    def __init__(self, fn: str):
        self.fn = fn
        self.ts = []

    def __call__(self, name, t, shape=None, dtype=None, optional=False):
        if t is None:
            if optional:
                return self
            raise ValueError(f"{self.fn}: {name} is required")
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{self.fn}: {name} must be a torch.Tensor")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{self.fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{self.fn}: {name} has dtype {t.dtype}, expected {dtype}")
        self.ts.append((name, t))
        return self

    def bytes(self, name, t, need: int):
        """A workspace: uint8, at least `need` bytes."""
        self(name, t, dtype=torch.uint8)
        if t.dim() != 1 or t.numel() < need:
            raise ValueError(f"{self.fn}: {name} holds {t.numel()} bytes, {need} needed")
        return self

    def done(self):
        dev = None
        for name, t in self.ts:
            if not t.is_cuda:
                raise ValueError(f"{self.fn}: {name} must be a device tensor")
            if not t.is_contiguous():
                raise ValueError(f"{self.fn}: {name} must be contiguous")
            if dev is None:
                dev = t.device
            elif t.device != dev:
                raise ValueError(f"{self.fn}: {name} is on {t.device}, the inputs on {dev}")


def _shape4(fn, P1):
    if not isinstance(P1, torch.Tensor) or P1.dim() != 4:
        raise ValueError(f"{fn}: P1 must be a [B, H, T, d_h] tensor")
    return tuple(P1.shape)


def fwd(P1, P2, V, tau, lam: float = 0.0, out=None, stream=None):
    """Y = relation forward of [B, H, T, d_h] device tensors; tau: float or [H]."""
    shp = _shape4("fwd", P1)
    B, H, T, D = shp
    a = _Args("fwd")("P1", P1)("P2", P2, shp, P1.dtype)("V", V, shp, P1.dtype)
    a("out", out, shp, P1.dtype, optional=True).done()
    if out is None:
        out = torch.empty_like(V)
    tau_keep, tau_p = _tau_arg(tau, H)
    st = lib().relation_fwd_ex(_ptr(P1), _ptr(P2), _ptr(V), tau_p, float(lam), _ptr(out),
                               B, H, T, D, _dtype_code(P1), _stream(stream))
    del tau_keep
    _check("relation_fwd_ex", st)
    return out


def fwd_lse(P1, P2, V, tau, lam: float = 0.0, out=None, lse=None, stream=None):
    """Training forward: (Y, LSE) with LSE the fp32 [B, H, T] row log normaliser."""
    shp = _shape4("fwd_lse", P1)
    B, H, T, D = shp
    a = _Args("fwd_lse")("P1", P1)("P2", P2, shp, P1.dtype)("V", V, shp, P1.dtype)
    a("out", out, shp, P1.dtype, optional=True)("lse", lse, (B, H, T), torch.float32, optional=True).done()
    if out is None:
        out = torch.empty_like(V)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=P1.device)
    tau_keep, tau_p = _tau_arg(tau, H)
    st = lib().relation_fwd_lse(_ptr(P1), _ptr(P2), _ptr(V), tau_p, float(lam), _ptr(out), _ptr(lse),
                                B, H, T, D, _dtype_code(P1), _stream(stream))
    del tau_keep
    _check("relation_fwd_lse", st)
    return out, lse


def bwd_workspace_bytes(B: int, H: int, T: int, d_h: int) -> int:
    return int(lib().relation_bwd_workspace_bytes(B, H, T, d_h))


def bwd_stored_workspace_bytes(B: int, H: int, T: int, d_h: int) -> int:
    return int(lib().relation_bwd_stored_workspace_bytes(B, H, T, d_h))


def bwd(P1, P2, V, tau, lam, Y, lse, dY, grads=None, workspace=None, stream=None, store_du=None):
    """Gradients (dP1, dP2, dV, dtau [H] fp32, dlambda [1] fp32) of sum(Y * dY),
    from the forward's inputs and its outputs Y, LSE (fwd_lse).

    store_du (when no workspace is given): True or None allocates the workspace
    with which the bf16 MFMA path stores dU (where that path exists), False
    the smaller one with which it recomputes the evidence for dP1."""
    shp = _shape4("bwd", P1)
    B, H, T, D = shp
    dt = P1.dtype
    a = _Args("bwd")("P1", P1)("P2", P2, shp, dt)("V", V, shp, dt)("Y", Y, shp, dt)("dY", dY, shp, dt)
    a("lse", lse, (B, H, T), torch.float32)
    if grads is not None:
        if len(grads) != 5:
            raise ValueError("bwd: grads must be (dP1, dP2, dV, dtau, dlam)")
        a("dP1", grads[0], shp, dt)("dP2", grads[1], shp, dt)("dV", grads[2], shp, dt)
        a("dtau", grads[3], (H,), torch.float32)("dlam", grads[4], (1,), torch.float32)
    need = bwd_workspace_bytes(B, H, T, D)
    if workspace is not None:
        a.bytes("workspace", workspace, need)
    elif store_du is not False and dt == torch.bfloat16:
        need = max(need, bwd_stored_workspace_bytes(B, H, T, D))
    a.done()
    if grads is None:
        grads = (torch.empty_like(P1), torch.empty_like(P2), torch.empty_like(V),
                 torch.empty(H, dtype=torch.float32, device=P1.device),
                 torch.empty(1, dtype=torch.float32, device=P1.device))
    dP1, dP2, dV, dtau, dlam = grads
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=P1.device)
    tau_keep, tau_p = _tau_arg(tau, H)
    st = lib().relation_bwd(_ptr(P1), _ptr(P2), _ptr(V), tau_p, float(lam), _ptr(Y), _ptr(lse), _ptr(dY),
                            _ptr(dP1), _ptr(dP2), _ptr(dV), _ptr(dtau), _ptr(dlam), B, H, T, D,
                            _dtype_code(P1), _ptr(workspace), workspace.numel(), _stream(stream))
    del tau_keep
    _check("relation_bwd", st)
    return dP1, dP2, dV, dtau, dlam


def _theta_arg(theta, H: int):
    if theta is None:
        return None, None
    arr = np.ascontiguousarray(np.asarray(theta, dtype=np.float32).reshape(-1))
    if arr.size != H // 2:
        raise ValueError(f"theta needs H/2 = {H // 2} angles")
    return arr, arr.ctypes.data_as(ctypes.POINTER(ctypes.c_float))


def _check_prestep(fn, P1, P2, I, pos0, out):
    shp = _shape4(fn, P1)
    a = _Args(fn)("P1", P1)("P2", P2, shp, P1.dtype)("I", I, shp, P1.dtype)
    a("pos0", pos0, (shp[0],), torch.int32, optional=True)
    if out is not None:
        if len(out) != 3:
            raise ValueError(f"{fn}: out must be (P1o, P2o, Io)")
        a("out[0]", out[0], shp, P1.dtype)("out[1]", out[1], shp, P1.dtype)("out[2]", out[2], shp, P1.dtype)
    a.done()
    return shp


def prestep(P1, P2, I, pos0=None, rope="interleaved", rope_base: float = 1e4, theta=None, pairing="A",
            out=None, stream=None):
    """RoPE on P1/P2 and Givens mixing of I ([B,H,T,d_h] device tensors); pos0:
    device int32[B] or None; theta: H/2 angles or None. out=(P1o, P2o, Io) may
    be the inputs themselves (in place)."""
    B, H, T, D = _check_prestep("prestep", P1, P2, I, pos0, out)
    if out is None:
        out = (torch.empty_like(P1), torch.empty_like(P2), torch.empty_like(I))
    th_keep, th_p = _theta_arg(theta, H)
    st = lib().relation_prestep(_ptr(P1), _ptr(P2), _ptr(I), _ptr(pos0), ROPE[rope], float(rope_base), th_p,
                                PAIRS[pairing], _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), B, H, T, D,
                                _dtype_code(P1), _stream(stream))
    del th_keep
    _check("relation_prestep", st)
    return out


def prestep_launcher(P1, P2, I, pos0, rope, rope_base, theta, pairing, out, stream=None):
    """relation_prestep with its arguments marshalled once: returns a callable
    that launches it again on the same tensors (for timing loops, where a
    short kernel would otherwise wait on the per-call marshalling)."""
    if out is None:
        raise ValueError("prestep_launcher: out is required")
    B, H, T, D = _check_prestep("prestep_launcher", P1, P2, I, pos0, out)
    th_keep, th_p = _theta_arg(theta, H)
    args = (_ptr(P1), _ptr(P2), _ptr(I), _ptr(pos0), ROPE[rope], float(rope_base), th_p, PAIRS[pairing],
            _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), B, H, T, D, _dtype_code(P1), _stream(stream))
    f = lib().relation_prestep

    def launch():
        _check("relation_prestep", f(*args))
        return th_keep

    return launch


def fwd_model(P1, P2, I, tau, lam: float = 0.0, pos0=None, rope="interleaved", rope_base: float = 1e4,
              theta=None, pairing="A", out=None, lse=None, workspace=None, stream=None):
    """The operator on raw projections: pre-steps, then the forward. Returns
    (Y, LSE or None, workspace): the workspace holds the pre-stepped P2 and I
    (second and third slots) and, unless the bf16 MFMA forward rotated P1
    itself, the rotated P1 (first slot)."""
    shp = _shape4("fwd_model", P1)
    B, H, T, D = shp
    a = _Args("fwd_model")("P1", P1)("P2", P2, shp, P1.dtype)("I", I, shp, P1.dtype)
    a("pos0", pos0, (B,), torch.int32, optional=True)("out", out, shp, P1.dtype, optional=True)
    a("lse", lse, (B, H, T), torch.float32, optional=True)
    need = int(lib().relation_fwd_model_workspace_bytes(B, H, T, D, _dtype_code(P1)))
    if workspace is not None:
        a.bytes("workspace", workspace, need)
    a.done()
    if out is None:
        out = torch.empty_like(I)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=P1.device)
    tau_keep, tau_p = _tau_arg(tau, H)
    th_keep, th_p = _theta_arg(theta, H)
    st = lib().relation_fwd_model(_ptr(P1), _ptr(P2), _ptr(I), _ptr(pos0), ROPE[rope], float(rope_base), th_p,
                                  PAIRS[pairing], tau_p, float(lam), _ptr(out), _ptr(lse), B, H, T, D,
                                  _dtype_code(P1), _ptr(workspace), workspace.numel(), _stream(stream))
    del tau_keep, th_keep
    _check("relation_fwd_model", st)
    return out, lse, workspace


def linear_fwd(P1, P2, I, alpha, tau, out=None, state=None, workspace=None, stream=None):
    """Linear Relation forward; alpha fp32 [B,H,T,d_h]; state: optional fp32
    [B,H,d_h,d_h] output for C_T. Returns (Y, state)."""
    shp = _shape4("linear_fwd", P1)
    B, H, T, D = shp
    a = _Args("linear_fwd")("P1", P1)("P2", P2, shp, P1.dtype)("I", I, shp, P1.dtype)
    a("alpha", alpha, shp, torch.float32)("out", out, shp, P1.dtype, optional=True)
    a("state", state, (B, H, D, D), torch.float32, optional=True)
    need = int(lib().relation_linear_workspace_bytes(B, H, T, D))
    if workspace is not None:
        a.bytes("workspace", workspace, need)
    a.done()
    if out is None:
        out = torch.empty_like(I)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=P1.device)
    tau_keep, tau_p = _tau_arg(tau, H)
    st = lib().relation_linear_fwd(_ptr(P1), _ptr(P2), _ptr(I), _ptr(alpha), tau_p, _ptr(out), _ptr(state),
                                   B, H, T, D, _dtype_code(P1), _ptr(workspace), workspace.numel(),
                                   _stream(stream))
    del tau_keep
    _check("relation_linear_fwd", st)
    return out, state


def decode_workspace_bytes(B: int, H: int, L_cap: int, d_h: int) -> int:
    return int(lib().relation_decode_workspace_bytes(B, H, L_cap, d_h))


def decode(p1, p2, v, cache_P2, cache_V, lens, tau, lam: float = 0.0, out=None,
           workspace=None, stream=None):
    """One Relation Cache decode step; p1/p2/v [B,H,d_h], caches [B,H,L_cap,d_h],
    lens int32[B] on the device."""
    if not isinstance(cache_P2, torch.Tensor) or cache_P2.dim() != 4:
        raise ValueError("decode: cache_P2 must be a [B, H, L_cap, d_h] tensor")
    B, H, L_cap, D = cache_P2.shape
    dt = cache_P2.dtype
    a = _Args("decode")("cache_P2", cache_P2)("cache_V", cache_V, cache_P2.shape, dt)
    a("p1", p1, (B, H, D), dt)("p2", p2, (B, H, D), dt)("v", v, (B, H, D), dt)("lens", lens, (B,), torch.int32)
    a("out", out, (B, H, D), dt, optional=True)
    need = decode_workspace_bytes(B, H, L_cap, D)
    if workspace is not None:
        a.bytes("workspace", workspace, need)
    a.done()
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=p1.device)
    if out is None:
        out = torch.empty_like(v)
    tau_keep, tau_p = _tau_arg(tau, H)
    st = lib().relation_decode(_ptr(p1), _ptr(p2), _ptr(v), _ptr(cache_P2), _ptr(cache_V),
                               _ptr(lens), tau_p, float(lam), _ptr(out), B, H, L_cap, D,
                               _dtype_code(p1), _ptr(workspace), workspace.numel(), _stream(stream))
    del tau_keep
    _check("relation_decode", st)
    return out


def decode_noalloc(p1, p2, v, cache_P2, cache_V, lens, tau, lam: float = 0.0, out=None, stream=None):
    """relation_decode_noalloc: decode with the library's scratch array for the
    partial states (no workspace; `out` must be given for a call that may not
    allocate)."""
    if not isinstance(cache_P2, torch.Tensor) or cache_P2.dim() != 4:
        raise ValueError("decode_noalloc: cache_P2 must be a [B, H, L_cap, d_h] tensor")
    B, H, L_cap, D = cache_P2.shape
    dt = cache_P2.dtype
    a = _Args("decode_noalloc")("cache_P2", cache_P2)("cache_V", cache_V, cache_P2.shape, dt)
    a("p1", p1, (B, H, D), dt)("p2", p2, (B, H, D), dt)("v", v, (B, H, D), dt)("lens", lens, (B,), torch.int32)
    a("out", out, (B, H, D), dt, optional=True).done()
    if out is None:
        out = torch.empty_like(v)
    tau_keep, tau_p = _tau_arg(tau, H)
    st = lib().relation_decode_noalloc(_ptr(p1), _ptr(p2), _ptr(v), _ptr(cache_P2), _ptr(cache_V), _ptr(lens),
                                       tau_p, float(lam), _ptr(out), B, H, L_cap, D, _dtype_code(p1),
                                       _stream(stream))
    del tau_keep
    _check("relation_decode_noalloc", st)
    return out


def cache_append(cache_P2, cache_V, lens, p2, v, stream=None):
    """Append the token's p2, v [B,H,d_h] at row lens[b] and increment lens."""
    if not isinstance(cache_P2, torch.Tensor) or cache_P2.dim() != 4:
        raise ValueError("cache_append: cache_P2 must be a [B, H, L_cap, d_h] tensor")
    B, H, L_cap, D = cache_P2.shape
    dt = cache_P2.dtype
    a = _Args("cache_append")("cache_P2", cache_P2)("cache_V", cache_V, cache_P2.shape, dt)
    a("lens", lens, (B,), torch.int32)("p2", p2, (B, H, D), dt)("v", v, (B, H, D), dt).done()
    st = lib().relation_cache_append(_ptr(cache_P2), _ptr(cache_V), _ptr(lens), _ptr(p2), _ptr(v),
                                     B, H, L_cap, D, _dtype_code(p2), _stream(stream))
    _check("relation_cache_append", st)


# ---- the paged Relation Cache ------------------------------------------------------
# These calls run in serving loops, where a step can be shorter than the checks of
# its arguments: the checks are one pass over (name, tensor, shape, dtype, dense).

_I32 = torch.int32


def _raw_stream(index: int) -> int:
    """The current stream of a device (torch.cuda.current_stream builds an object
    around it first, 3 us)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _heads_contiguous(t, shape) -> bool:
    st = t.stride()
    return st[2] == 1 and (shape[1] <= 1 or st[1] == shape[2])


def _check_tensors(fn, specs):
    """Shapes, dtypes and token layouts of all tensors, their device and contiguity. dense
    False: a packed token tensor [N, heads, d_h] whose tokens may be further apart (a slice of
    a fused projection). Returns the device. One pass where nothing is wrong; what is
    wrong is told by _refuse."""
    first = specs[0][1]
    if isinstance(first, torch.Tensor) and first.is_cuda:
        index = first.get_device()
        for _, t, shape, dtype, dense in specs:
            if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.get_device() == index
                    and (t.is_contiguous() if dense else _heads_contiguous(t, shape))):
                break
        else:
            return first.device
    return _refuse(fn, specs)


def _refuse(fn, specs):
    """Shapes, dtypes and token layouts of all tensors first, whatever device they
    are on; then device and contiguity."""
    for name, t, shape, dtype, dense in specs:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{fn}: {name} must be a torch.Tensor")
        if t.shape != shape:
            raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype is not dtype:
            raise TypeError(f"{fn}: {name} has dtype {t.dtype}, expected {dtype}")
        if not dense and not _heads_contiguous(t, shape):
            raise ValueError(f"{fn}: the heads of each token of {name} must be contiguous")
    dev = specs[0][1].device
    if dev.type != "cuda":
        raise ValueError(f"{fn}: {specs[0][0]} must be a device tensor")
    for name, t, _, _, dense in specs:
        if t.device != dev:
            raise ValueError(f"{fn}: {name} is on {t.device}, the inputs on {dev}")
        if dense and not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be contiguous")
    raise AssertionError(fn)


def _run_on(fn, dev, stream, args):
    """The library call fn(*args, stream) with the tensors' device current, on the
    caller's stream (which has to be of that device) or the current one."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"{fn}: the stream is on {stream.device}, the tensors on {dev}")
    f = getattr(lib(), fn)
    sp = _raw_stream(dev.index) if stream is None else stream.cuda_stream
    if dev.index == torch.cuda.current_device():
        st = f(*args, sp)
    else:
        with torch.cuda.device(dev):
            st = f(*args, sp)
    if st != 0:
        raise RelationError(fn, st)


def _on(stream):
    """Where a call allocates: its stream's memory, which later work of other
    streams does not reuse before the call has run."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _count(name: str, x) -> int:
    x = int(x)
    if not -2**31 <= x < 2**31:
        raise ValueError(f"{name} = {x} does not fit 32 bits")
    return x


def _host_floats(x, n: int, c_type=ctypes.c_float):
    """Host float[n] (double[n]) from a float or n of them."""
    if isinstance(x, (list, tuple)) and len(x) == n:
        return (c_type * n)(*x)
    if isinstance(x, float):
        return (c_type * n)(*([x] * n))
    arr = np.ascontiguousarray(np.broadcast_to(np.asarray(x, dtype=c_type), (n,)))
    return (c_type * n).from_buffer_copy(arr)


def _pages(fn, cache_P2):
    if not isinstance(cache_P2, torch.Tensor) or cache_P2.dim() != 4:
        raise ValueError(f"{fn}: cache_P2 must be a [n_pages, H_kv, page_size, d_h] tensor")
    return cache_P2.shape


def _tokens(fn, name, t):
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{fn}: {name} must be an [N, heads, d_h] tensor")
    return t.shape


def _table(fn, t):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{fn}: block_table must be an [S, max_pages] tensor")
    _count("max_pages", t.shape[1])
    return t.shape


def _token_dtype(fn, specs, cdt, shp, scale):
    """The tokens' type for pages of type cdt; 8-bit pages have scales, which join specs."""
    if cdt is torch.float8_e4m3fn:
        specs.append(("scale", scale, (shp[0], shp[1], 2, shp[2]), torch.float8_e8m0fnu, True))
        return torch.bfloat16
    if scale is not None:
        raise TypeError(f"{fn}: scale belongs to float8_e4m3fn pages, these are {cdt}")
    return cdt


def _ld(t) -> int:
    """Elements between consecutive tokens of a packed [N, heads, d_h] tensor."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def page_map(lens, n_new, block_table, free_pages, n_free, N: int, page_size: int, n_pages: int, out=None,
             stream=None):
    """Block table, slots and positions of a packed batch of N token rows, from
    the request lengths: lens, n_new int32[S] (n_new -1: finished, its pages
    return to the list), block_table int32[S, max_pages] and free_pages int32[F]
    (both updated in place), n_free int32[1]. Returns (cu [S+1], total [S], slot
    [N], pos [N], n_free_out [1]); out: the five tensors (n_free_out may be n_free)."""
    fn = "page_map"
    S, width = _table(fn, block_table)
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("page_map: free_pages must be a 1-d tensor")
    N, F = _count("N", N), _count("F", free_pages.shape[0])
    page_size, n_pages = _count("page_size", page_size), _count("n_pages", n_pages)
    specs = [("block_table", block_table, (S, width), _I32, True), ("free_pages", free_pages, (F,), _I32, True),
             ("lens", lens, (S,), _I32, True), ("n_new", n_new, (S,), _I32, True), ("n_free", n_free, (1,), _I32, True)]
    if out is not None:
        if len(out) != 5:
            raise ValueError("page_map: out must be (cu, total, slot, pos, n_free_out)")
        cu, total, slot, pos, n_free_out = out
        specs += [("cu", cu, (S + 1,), _I32, True), ("total", total, (S,), _I32, True), ("slot", slot, (N,), _I32, True),
                  ("pos", pos, (N,), _I32, True), ("n_free_out", n_free_out, (1,), _I32, True)]
    dev = _check_tensors(fn, specs)
    if out is None:
        with _on(stream):
            out = tuple(torch.empty(max(n, 0), dtype=_I32, device=dev) for n in (S + 1, S, N, N, 1))
        cu, total, slot, pos, n_free_out = out
    _run_on("relation_page_map", dev, stream,
            (lens.data_ptr(), n_new.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(), n_free.data_ptr(),
             n_free_out.data_ptr(), cu.data_ptr(), total.data_ptr(), slot.data_ptr(), pos.data_ptr(), S, N, F, width,
             page_size, n_pages))
    return out


def paged_append(P2, I, slot, cache_P2, cache_V, P1=None, pos=None, rope="none", rope_base: float = 1e4, theta=None,
                 pairing="A", out=None, stream=None, scale=None):
    """Pre-steps of a packed batch with P2 and the mixed I stored into the pages:
    P2, I [N, H_kv, d_h] and optionally P1 [N, H, d_h] (tokens may be slices of a
    fused projection), slot and pos int32[N] (page_map, tree_plan), caches [n_pages,
    H_kv, page_size, d_h]. Returns the rotated P1 ([N, H, d_h]; out, which may be P1
    itself if contiguous) or None. Rows of tokens without a slot are not written
    (zero in a P1 that the call allocates).

    8-bit pages: float8_e4m3fn caches with scale, float8_e8m0fnu [n_pages, H_kv, 2,
    page_size] (of the P2 and the V rows), and bfloat16 tokens, quantised as they are
    stored."""
    fn = "paged_append"
    n_pages, Hkv, ps, D = shp = _pages(fn, cache_P2)
    N = _tokens(fn, "P2", P2)[0]
    cdt, H = cache_P2.dtype, 0
    specs = [("cache_P2", cache_P2, shp, cdt, True), ("cache_V", cache_V, shp, cdt, True)]
    dt = _token_dtype(fn, specs, cdt, shp, scale)
    specs += [("P2", P2, (N, Hkv, D), dt, False), ("I", I, (N, Hkv, D), dt, False), ("slot", slot, (N,), _I32, True)]
    if pos is not None:
        specs.append(("pos", pos, (N,), _I32, True))
    if P1 is not None:
        H = _tokens(fn, "P1", P1)[1]
        specs.append(("P1", P1, (N, H, D), dt, False))
        if out is not None:
            specs.append(("out", out, (N, H, D), dt, True))
    elif out is not None:
        raise ValueError("paged_append: out is given without P1")
    dev = _check_tensors(fn, specs)
    if theta is not None and len(theta) != Hkv // 2:
        raise ValueError(f"theta needs H_kv/2 = {Hkv // 2} angles")
    if P1 is not None and out is None:
        with _on(stream):
            out = torch.zeros((N, H, D), dtype=dt, device=dev)
    name, pages, angle = "relation_paged_append", (), ctypes.c_float
    if scale is not None:
        name, pages, angle = "relation_paged_append_q8", (scale.data_ptr(),), ctypes.c_double
    _run_on(name, dev, stream,
            (_ptr(P1), P2.data_ptr(), I.data_ptr(), 0 if P1 is None else _ld(P1), _ld(P2), _ld(I), slot.data_ptr(),
             _ptr(pos), ROPE[rope], float(rope_base), None if theta is None else _host_floats(theta, Hkv // 2, angle),
             PAIRS[pairing], _ptr(out), cache_P2.data_ptr(), cache_V.data_ptr(), *pages, N, H, Hkv, D, n_pages, ps,
             *(() if pages else (_dtype_code(cache_P2),))))
    return out


def paged_workspace_bytes(N: int, S: int, H: int, H_kv: int, d_h: int) -> int:
    return int(lib().relation_paged_workspace_bytes(N, S, H, H_kv, d_h))


def paged_fwd(P1, cache_P2, cache_V, block_table, total, cu, tau, lam: float = 0.0, max_new=None, out=None,
              workspace=None, stream=None, scale=None, tree=None):
    """Y [N, H, d_h] of a packed batch of new tokens whose own rows are in the
    pages already: P1 [N, H, d_h] (rotated), caches [n_pages, H_kv, page_size,
    d_h], block_table int32[S, max_pages], total int32[S], cu int32[S+1]
    (page_map). max_new: the most new tokens of one request (default N; the closer,
    the better the choice of kernels). Rows that no request owns are not written (zero
    in a Y that the call allocates).

    8-bit pages: float8_e4m3fn caches with scale (paged_append) and a bfloat16 P1.
    tree: int32[N, words] ancestor bits (tree_plan): a token of a request of at most
    32 * words new tokens sees, of those, its ancestors and itself alone."""
    fn = "paged_fwd"
    n_pages, Hkv, ps, D = shp = _pages(fn, cache_P2)
    N, H = _tokens(fn, "P1", P1)[:2]
    S, width = _table(fn, block_table)
    cdt = cache_P2.dtype
    specs = [("cache_P2", cache_P2, shp, cdt, True), ("cache_V", cache_V, shp, cdt, True)]
    dt = _token_dtype(fn, specs, cdt, shp, scale)
    specs += [("P1", P1, (N, H, D), dt, False),
              ("block_table", block_table, (S, width), _I32, True), ("total", total, (S,), _I32, True),
              ("cu", cu, (S + 1,), _I32, True)]
    words = 0
    if tree is not None:
        words = _tree_words(fn, tree)
        specs.append(("tree", tree, (N, words), _I32, True))
    if out is not None:
        specs.append(("out", out, (N, H, D), dt, True))
    need = paged_workspace_bytes(N, S, H, Hkv, D)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or workspace.dim() != 1:
            raise TypeError("paged_fwd: workspace must be a 1-d torch.uint8 tensor")
        if workspace.numel() < need:
            raise ValueError(f"paged_fwd: workspace holds {workspace.numel()} bytes, {need} needed")
        specs.append(("workspace", workspace, workspace.shape, torch.uint8, True))
    max_new = N if max_new is None else _count("max_new", max_new)
    dev = _check_tensors(fn, specs)
    if out is None or workspace is None:
        with _on(stream):
            if out is None:
                out = torch.zeros((N, H, D), dtype=dt, device=dev)
            if workspace is None:
                workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    args = (block_table.data_ptr(), total.data_ptr(), cu.data_ptr())
    if scale is None and tree is None:
        fn, args, pages = "relation_paged_fwd", args, _dtype_code(P1)
    else:
        fn, args = "relation_paged_fwd_ex", (_ptr(scale), *args, _ptr(tree), words)
        pages = REL_E4M3 if scale is not None else _dtype_code(P1)
    _run_on(fn, dev, stream,
            (P1.data_ptr(), _ld(P1), cache_P2.data_ptr(), cache_V.data_ptr(), *args, _host_floats(tau, H), float(lam),
             out.data_ptr(), N, S, H, Hkv, D, n_pages, ps, width, max_new, pages, workspace.data_ptr(),
             workspace.numel()))
    return out


# ---- trees of drafted tokens -------------------------------------------------------

MAX_TREE_WORDS = 32


def _tree_words(fn, tree) -> int:
    if not isinstance(tree, torch.Tensor) or tree.dim() != 2 or not 1 <= tree.shape[1] <= MAX_TREE_WORDS:
        raise ValueError(f"{fn}: tree must be an [N, words] tensor of 1 to {MAX_TREE_WORDS} words")
    return tree.shape[1]


def tree_plan(parent, total, cu, words: int, out=None, stream=None):
    """Ancestor bits and positions of packed trees of drafted tokens: parent int32[N],
    each token's parent as its place among its request's new tokens (outside [0, own
    place): a root), total int32[S], cu int32[S+1] (page_map). Requests of more than
    32 * words new tokens are chunks, each token seeing all before it. Returns (tree
    [N, words], pos [N]) int32; out: the two tensors. Rows of tree that no tree's token
    owns are not written (zero in a tree that the call allocates)."""
    fn = "tree_plan"
    for name, t in (("parent", parent), ("total", total)):
        if not isinstance(t, torch.Tensor) or t.dim() != 1:
            raise ValueError(f"{fn}: {name} must be a 1-d tensor")
    N, S, words = _count("N", parent.shape[0]), total.shape[0], int(words)
    if not 1 <= words <= MAX_TREE_WORDS:
        raise ValueError(f"{fn}: words must be 1 to {MAX_TREE_WORDS}, not {words}")
    specs = [("parent", parent, (N,), _I32, True), ("total", total, (S,), _I32, True), ("cu", cu, (S + 1,), _I32, True)]
    if out is not None:
        if len(out) != 2:
            raise ValueError(f"{fn}: out must be (tree, pos)")
        specs += [("tree", out[0], (N, words), _I32, True), ("pos", out[1], (N,), _I32, True)]
    dev = _check_tensors(fn, specs)
    if out is None:
        with _on(stream):
            out = (torch.zeros((N, words), dtype=_I32, device=dev), torch.empty(N, dtype=_I32, device=dev))
    _run_on("relation_tree_plan", dev, stream,
            (parent.data_ptr(), total.data_ptr(), cu.data_ptr(), out[0].data_ptr(), out[1].data_ptr(), N, S, words))
    return out


def paged_keep(cache_P2, cache_V, block_table, total, cu, keep, n_keep, lens, free_pages, n_free, n_free_out=None,
               scale=None, stream=None):
    """Cuts each request back to the new tokens that it keeps: request b keeps n_keep[b]
    (int32[S]), whose places among its new tokens keep[cu[b]:] (int32[N]) names in
    growing order. Their rows move to the front of the new ones (caches, and scale for
    float8_e4m3fn ones, in place), lens int32[S] becomes the cached rows, and the pages
    behind them go back to free_pages int32[F] (n_free int32[1] entries). Returns the
    list's new count, int32[1] (n_free_out, which may be n_free)."""
    fn = "paged_keep"
    n_pages, Hkv, ps, D = shp = _pages(fn, cache_P2)
    S, width = _table(fn, block_table)
    for name, t in (("keep", keep), ("free_pages", free_pages)):
        if not isinstance(t, torch.Tensor) or t.dim() != 1:
            raise ValueError(f"{fn}: {name} must be a 1-d tensor")
    N, F = _count("N", keep.shape[0]), _count("F", free_pages.shape[0])
    cdt = cache_P2.dtype
    specs = [("cache_P2", cache_P2, shp, cdt, True), ("cache_V", cache_V, shp, cdt, True)]
    _token_dtype(fn, specs, cdt, shp, scale)
    specs += [("block_table", block_table, (S, width), _I32, True), ("total", total, (S,), _I32, True),
              ("cu", cu, (S + 1,), _I32, True), ("keep", keep, (N,), _I32, True), ("n_keep", n_keep, (S,), _I32, True),
              ("lens", lens, (S,), _I32, True), ("free_pages", free_pages, (F,), _I32, True),
              ("n_free", n_free, (1,), _I32, True)]
    if n_free_out is not None:
        specs.append(("n_free_out", n_free_out, (1,), _I32, True))
    pages = REL_E4M3 if cdt is torch.float8_e4m3fn else _dtype_code(cache_P2)
    dev = _check_tensors(fn, specs)
    if n_free_out is None:
        with _on(stream):
            n_free_out = torch.empty(1, dtype=_I32, device=dev)
    _run_on("relation_paged_keep", dev, stream,
            (cache_P2.data_ptr(), cache_V.data_ptr(), _ptr(scale), block_table.data_ptr(), total.data_ptr(), cu.data_ptr(),
             keep.data_ptr(), n_keep.data_ptr(), lens.data_ptr(), free_pages.data_ptr(), n_free.data_ptr(),
             n_free_out.data_ptr(), N, S, F, Hkv, D, n_pages, ps, width, pages))
    return n_free_out
