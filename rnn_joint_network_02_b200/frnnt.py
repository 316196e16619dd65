"""Thin Python binding of libfrnnt.so (ctypes).

Argument marshalling only: every step of the forward and backward pass runs
in the library's CUDA kernels.  PyTorch supplies device memory and the
stream.  If the shared library is missing the first call raises; there is no
other implementation behind these names.
"""

from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfrnnt.so")

UNTILED, TILED = 0, 1
F32, BF16 = 0, 1
PATH_AUTO, PATH_SIMT = 0, 1

OK = 0
STATUS_LENGTH, STATUS_LABEL, STATUS_TIMEOUT, STATUS_BOUNDS, STATUS_INDEX = 1, 2, 4, 8, 16

EXPORTED = ("frnnt_workspace_size", "frnnt_fwd_bwd", "frnnt_error_string", "frnnt_version", "frnnt_profile",
            "frnnt_profile_read", "frnnt_fwd_bwd_noalloc", "frnnt_fwd_bwd_pruned", "frnnt_fwd_bwd_tdt",
            "frnnt_token_logprobs", "frnnt_token_logprobs_bwd", "frnnt_recurrence_fwd", "frnnt_recurrence_bwd",
            "frnnt_recurrence_step", "frnnt_dropout")
MAX_DURATIONS = 8
MAX_TOKENS, MAX_TOP, NO_TOKEN, SCAN_CHUNK = 32, 32, -1, 128
NOALLOC_MAX_BYTES = 64 * 1024 * 1024
TEST_HOOKS = ("frnnt_test_gemm_bf16", "frnnt_test_joint_variant", "frnnt_test_lose_gemm_loads",
              "frnnt_test_lose_scan_maps", "frnnt_test_refuse_clusters")


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("U", ctypes.c_int), ("D_enc", ctypes.c_int),
                ("D_pred", ctypes.c_int), ("H", ctypes.c_int), ("V", ctypes.c_int), ("blank", ctypes.c_int),
                ("dtype", ctypes.c_int), ("mode", ctypes.c_int), ("path", ctypes.c_int),
                ("chunk_cells", ctypes.c_int), ("loss", ctypes.c_int), ("prune_S", ctypes.c_int),
                ("n_dur", ctypes.c_int), ("durations", ctypes.c_int * 8), ("wgrad_f32", ctypes.c_int)]


class LogprobDims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("V", ctypes.c_int), ("K", ctypes.c_int), ("top", ctypes.c_int),
                ("dtype", ctypes.c_int), ("ld", ctypes.c_longlong), ("ldd", ctypes.c_longlong),
                ("lse_rest", ctypes.c_void_p)]


class RecurrenceDims(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_int) for k in ("B", "T", "D", "dtype")] +
                [(f"{k}_{s}", ctypes.c_longlong) for k in ("x", "gate", "h", "dh", "dx", "dgate") for s in ("sb", "st")])


class StepDims(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_int) for k in ("N", "S", "D", "dtype")] +
                [("x_sn", ctypes.c_longlong), ("gate_sn", ctypes.c_longlong)])


class DropoutDims(ctypes.Structure):
    _fields_ = [("R", ctypes.c_longlong), ("C", ctypes.c_longlong), ("dtype", ctypes.c_int),
                ("x_ld", ctypes.c_longlong), ("y_ld", ctypes.c_longlong), ("p", ctypes.c_double),
                ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64)]


class StageStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int), ("calls", ctypes.c_int),
                ("ms", ctypes.c_double)]


class FrnntError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"frnnt error {code}: {msg}")
        self.code = code


class FrnntStatusError(RuntimeError):
    def __init__(self, bits: int):
        names = [n for n, v in (("invalid lengths", STATUS_LENGTH), ("invalid labels", STATUS_LABEL),
                                ("a bounded device wait timed out", STATUS_TIMEOUT),
                                ("invalid pruning bounds", STATUS_BOUNDS),
                                ("invalid parent rows", STATUS_INDEX))
                 if bits & v]
        super().__init__(f"frnnt device status {bits}: {'; '.join(names)}")
        self.bits = bits


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded shared library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m rnn_joint_network_02_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32p, f32p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
        L.frnnt_workspace_size.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(ctypes.c_size_t)]
        L.frnnt_workspace_size.restype = ctypes.c_int
        L.frnnt_fwd_bwd.argtypes = ([ctypes.POINTER(Dims)] + [vp] * 6 + [i32p] * 3 + [f32p, f32p] + [vp] * 6 +
                                    [vp, ctypes.c_size_t, i32p, vp])
        L.frnnt_fwd_bwd.restype = ctypes.c_int
        L.frnnt_fwd_bwd_pruned.argtypes = ([ctypes.POINTER(Dims)] + [vp] * 6 + [i32p] * 4 + [f32p, f32p] + [vp] * 6 +
                                           [vp, ctypes.c_size_t, i32p, vp])
        L.frnnt_fwd_bwd_pruned.restype = ctypes.c_int
        L.frnnt_fwd_bwd_tdt.argtypes = ([ctypes.POINTER(Dims)] + [vp] * 8 + [i32p] * 3 + [f32p, f32p] + [vp] * 8 +
                                        [vp, ctypes.c_size_t, i32p, vp])
        L.frnnt_fwd_bwd_tdt.restype = ctypes.c_int
        L.frnnt_fwd_bwd_noalloc.argtypes = ([ctypes.POINTER(Dims)] + [vp] * 6 + [i32p] * 3 + [f32p, f32p] +
                                            [vp] * 6 + [i32p, vp])
        L.frnnt_fwd_bwd_noalloc.restype = ctypes.c_int
        L.frnnt_error_string.argtypes = [ctypes.c_int]
        L.frnnt_error_string.restype = ctypes.c_char_p
        L.frnnt_version.argtypes = []
        L.frnnt_version.restype = ctypes.c_char_p
        L.frnnt_profile.argtypes = [ctypes.c_int]
        L.frnnt_profile.restype = ctypes.c_int
        L.frnnt_profile_read.argtypes = [ctypes.POINTER(StageStat), ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
        L.frnnt_profile_read.restype = ctypes.c_int
        L.frnnt_token_logprobs.argtypes = [ctypes.POINTER(LogprobDims)] + [vp] * 9
        L.frnnt_token_logprobs_bwd.argtypes = [ctypes.POINTER(LogprobDims)] + [vp] * 11
        L.frnnt_recurrence_fwd.argtypes = [ctypes.POINTER(RecurrenceDims)] + [vp] * 9
        L.frnnt_recurrence_bwd.argtypes = [ctypes.POINTER(RecurrenceDims)] + [vp] * 11
        L.frnnt_recurrence_step.argtypes = [ctypes.POINTER(StepDims)] + [vp] * 9
        L.frnnt_dropout.argtypes = [ctypes.POINTER(DropoutDims)] + [vp] * 4
        for name in ("frnnt_token_logprobs", "frnnt_token_logprobs_bwd", "frnnt_recurrence_fwd",
                     "frnnt_recurrence_bwd", "frnnt_recurrence_step", "frnnt_dropout"):
            getattr(L, name).restype = ctypes.c_int
        L.frnnt_test_gemm_bf16.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, ctypes.c_int,
                                           ctypes.c_longlong, vp, ctypes.c_int, ctypes.c_longlong, ctypes.c_int,
                                           ctypes.c_int, vp, ctypes.c_longlong, ctypes.c_int, vp, vp]
        L.frnnt_test_gemm_bf16.restype = ctypes.c_int
        L.frnnt_test_joint_variant.argtypes = [ctypes.c_int]
        L.frnnt_test_joint_variant.restype = ctypes.c_int
        L.frnnt_test_lose_gemm_loads.argtypes = [ctypes.c_int]
        L.frnnt_test_lose_gemm_loads.restype = ctypes.c_int
        L.frnnt_test_lose_scan_maps.argtypes = [ctypes.c_int] * 4
        L.frnnt_test_lose_scan_maps.restype = ctypes.c_int
        L.frnnt_test_refuse_clusters.argtypes = [ctypes.c_int]
        L.frnnt_test_refuse_clusters.restype = ctypes.c_int
        _lib = L
    return _lib


def error_string(code: int) -> str:
    return lib().frnnt_error_string(code).decode()


def version() -> str:
    return lib().frnnt_version().decode()


def profile(enable: bool) -> None:
    """Per-stage CUDA-event timing on/off for later calls (launch counts are always kept)."""
    lib().frnnt_profile(1 if enable else 0)


def profile_read() -> dict:
    """{stage: dict(launches, calls, ms)} accumulated since the previous read (then reset)."""
    cap = 64
    arr = (StageStat * cap)()
    n = ctypes.c_int(0)
    rc = lib().frnnt_profile_read(arr, cap, ctypes.byref(n))
    if rc != OK:
        raise FrnntError(rc, error_string(rc))
    out = {}
    for i in range(min(n.value, cap)):
        st = arr[i]
        if st.calls or st.launches:
            out[st.name.decode()] = dict(launches=st.launches, calls=st.calls, ms=st.ms)
    return out


LOSSES = {"marginal": 0, "viterbi": 1}


def make_dims(B, T, U, D_enc, D_pred, H, V, dtype="bf16", mode="tiled", path="auto", chunk_cells=0,
              blank=0, loss="marginal", prune_S=0, durations=(), wgrad_f32=False) -> Dims:
    """``durations`` (token-and-duration transducer): the duration set, or () for the transducer.
    ``wgrad_f32``: weight gradients come back as the library's fp32 accumulators."""
    if len(durations) > MAX_DURATIONS:
        raise ValueError(f"at most {MAX_DURATIONS} durations")
    dur = (ctypes.c_int * 8)(*[int(x) for x in durations])
    return Dims(B, T, U, D_enc, D_pred, H, V, blank, BF16 if dtype == "bf16" else F32,
                TILED if mode == "tiled" else UNTILED, PATH_SIMT if path == "simt" else PATH_AUTO,
                chunk_cells, LOSSES[loss], prune_S, len(durations), dur, 1 if wgrad_f32 else 0)


def workspace_size(dims: Dims) -> int:
    n = ctypes.c_size_t(0)
    rc = lib().frnnt_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != OK:
        raise FrnntError(rc, error_string(rc))
    return n.value


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def dims_of(f, g, W_o, dtype, mode, path, chunk_cells, blank, loss="marginal", prune_S=0, durations=(),
            wgrad_f32=False) -> Dims:
    B, T, D_enc = f.shape
    U = g.shape[1] - 1
    V, H = W_o.shape
    return make_dims(B, T, U, D_enc, g.shape[2], H, V, dtype, mode, path, chunk_cells, blank, loss, prune_S,
                     durations, wgrad_f32)


def _check_call(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss, out, bounds=None, W_d=None, b_d=None,
                wgrad_f32=False):
    """Host-side checks before any pointer reaches the library: a tensor of the
    wrong shape, dtype, layout or device would otherwise be read or written out
    of bounds by the kernels.  Shapes and dtypes are checked first, then that
    every tensor lives on the same CUDA device.  Raises ValueError."""
    if f.dim() != 3 or g.dim() != 3 or W_o.dim() != 2:
        raise ValueError("f must be [B, T, D_enc], g [B, U+1, D_pred] and W_o [V, H]")
    B, T, D_enc = f.shape
    Up1, D_pred = g.shape[1], g.shape[2]
    V, H = W_o.shape
    ft = f.dtype
    if ft not in (torch.float32, torch.bfloat16):
        raise ValueError(f"f must be float32 or bfloat16, not {ft}")
    want = [("f", f, (B, T, D_enc), ft), ("g", g, (B, Up1, D_pred), ft), ("W_f", W_f, (D_enc, H), ft),
            ("W_g", W_g, (D_pred, H), ft), ("W_o", W_o, (V, H), ft), ("b_o", b_o, (V,), ft),
            ("labels", labels, (B, Up1 - 1), torch.int32), ("T_len", T_len, (B,), torch.int32),
            ("U_len", U_len, (B,), torch.int32)]
    if grad_loss is not None:
        want.append(("grad_loss", grad_loss, (B,), torch.float32))
    if bounds is not None:
        want.append(("bounds", bounds, (B, T), torch.int32))
    if W_d is not None or b_d is not None:
        if W_d is None or b_d is None or W_d.dim() != 2:
            raise ValueError("the duration head needs W_d [n_dur, H] and b_d [n_dur]")
        want += [("W_d", W_d, (W_d.shape[0], H), ft), ("b_d", b_d, (W_d.shape[0],), ft)]
    if out is not None:
        wt = torch.float32 if wgrad_f32 else ft     # dtype of the weight gradients
        want += [("out.loss", out.loss, (B,), torch.float32), ("out.df", out.df, tuple(f.shape), ft),
                 ("out.dg", out.dg, tuple(g.shape), ft), ("out.dW_f", out.dW_f, (D_enc, H), wt),
                 ("out.dW_g", out.dW_g, (D_pred, H), wt), ("out.dW_o", out.dW_o, (V, H), wt),
                 ("out.db_o", out.db_o, (V,), wt), ("out.status", out.status, (4,), torch.int32)]
        if W_d is not None:
            if out.dW_d is None or out.db_d is None:
                raise ValueError("out has no duration-head gradients")
            want += [("out.dW_d", out.dW_d, tuple(W_d.shape), wt), ("out.db_d", out.db_d, tuple(b_d.shape), wt)]
    for name, t, shape, dt in want:
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype != dt:
            raise ValueError(f"{name} is {t.dtype}, expected {dt}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if f.device.type != "cuda":
        raise ValueError("the library computes on the GPU: pass CUDA tensors")
    for name, t, _, _ in want:
        if t.device != f.device:
            raise ValueError(f"{name} is on {t.device}, the call's tensors on {f.device}")
    if out is not None and out.workspace is not None and out.workspace.device != f.device:
        raise ValueError(f"the workspace is on {out.workspace.device}, the call's tensors on {f.device}")


class Outputs:
    """Preallocated outputs and workspace of one call shape.

    With ``dims.wgrad_f32`` the weight gradients (dW_f, dW_g, dW_o, db_o and
    the duration head's dW_d, db_d) are fp32 views into one flat buffer,
    ``wflat``, so a data-parallel exchange sums them with one all-reduce."""

    def __init__(self, f, g, W_f, W_g, W_o, b_o, dims: Dims, with_workspace: bool = True, W_d=None, b_d=None):
        dev = f.device
        self.loss = torch.empty(f.shape[0], dtype=torch.float32, device=dev)
        self.df = torch.empty_like(f)
        self.dg = torch.empty_like(g)
        weights = [("dW_f", W_f), ("dW_g", W_g), ("dW_o", W_o), ("db_o", b_o)]
        if W_d is not None:
            weights += [("dW_d", W_d), ("db_d", b_d)]
        self.dW_d = self.db_d = None
        self.wflat = None
        self.dropped = None      # f and g after dropout, once a call with dropout has needed them
        if dims.wgrad_f32:
            # segments start on 16-byte boundaries (the library's alignment rule)
            sizes = [(t.numel() + 3) // 4 * 4 for _, t in weights]
            self.wflat = torch.zeros(sum(sizes), dtype=torch.float32, device=dev)
            off = 0
            for (name, t), n in zip(weights, sizes):
                setattr(self, name, self.wflat[off:off + t.numel()].view(t.shape))
                off += n
        else:
            for name, t in weights:
                setattr(self, name, torch.empty_like(t))
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        n = max(workspace_size(dims), 16) if with_workspace else 16
        self.workspace = torch.empty(n, dtype=torch.uint8, device=dev)

    def grads(self):
        d = dict(df=self.df, dg=self.dg, dW_f=self.dW_f, dW_g=self.dW_g, dW_o=self.dW_o, db_o=self.db_o)
        if self.dW_d is not None:
            d.update(dW_d=self.dW_d, db_d=self.db_d)
        return d


class Dropout(NamedTuple):
    """Dropout of a loss call's inputs f and g (the ``dropout`` argument of
    fwd_bwd and its variants): each entry is dropped with probability p before
    the joint network and the rest scaled by 1 / (1 - p), and df and dg are the
    gradients for the f and g that were passed.  The mask comes from
    ``dropout`` (below) and is never stored: f's entries take the counters from
    ``offset`` on, g's those that follow.  A new call needs new numbers: another
    ``seed``, or ``offset`` moved on by ``counters(f, g)``; ``seed`` may be a
    device tensor (captured graphs).  Data-parallel ranks need a seed each.
    f and g, and df and dg, are scaled in fp32 and rounded to their type once
    more than in a call without dropout (the joint network takes and gives that
    type)."""
    p: float
    seed: "int | torch.Tensor"
    offset: int = 0

    @staticmethod
    def counters(f, g) -> int:
        """Counters that one call uses."""
        return (f.numel() + 7) // 8 + (g.numel() + 7) // 8


def _with_dropout(drop, f, g, out, call):
    """``call(f, g)`` on the dropped inputs, its df and dg masked alike, all on the current stream."""
    if out is not None and out.dropped is None:
        out.dropped = (torch.empty_like(f), torch.empty_like(g))
    fd, gd = (None, None) if out is None else out.dropped
    at = (drop.offset, drop.offset + (f.numel() + 7) // 8)
    loss, grads = call(dropout(f, drop.p, drop.seed, at[0], fd), dropout(g, drop.p, drop.seed, at[1], gd))
    dropout(grads["df"], drop.p, drop.seed, at[0], grads["df"])
    dropout(grads["dg"], drop.p, drop.seed, at[1], grads["dg"])
    return loss, grads


def _loss_place(dev, stream):
    """The context that a loss call is made in (see _elsewhere), so that the
    buffers it allocates belong to its stream and its status is read there; None
    where the stream that is given is the current one."""
    if stream is not None and _raw_stream and stream.device == dev and _current_device() == dev.index and \
            stream.cuda_stream == _raw_stream(dev.index):
        return None
    return _elsewhere(dev, stream)


def fwd_bwd(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss=None, mode="tiled", path="auto",
            chunk_cells=0, blank=0, out: Outputs | None = None, check=True, stream=None, loss="marginal",
            wgrad_f32=False, dropout: Dropout | None = None):
    """One call of frnnt_fwd_bwd on CUDA tensors.

    Float tensors are all float32 or all bfloat16; labels/T_len/U_len int32.
    ``loss`` is "marginal" (every alignment) or "viterbi" (the best one).
    ``wgrad_f32``: the weight gradients come back in fp32 (unrounded).
    ``dropout``: of f and g, see Dropout.
    ``stream``: the work is queued there instead of on the current stream, and
    what the call allocates belongs to it.
    Returns (loss [B] fp32, dict of gradients).  With ``check`` the device
    status word is read back (one 4-byte device-to-host copy, which
    synchronises the stream) and a non-zero status raises FrnntStatusError.
    """
    _check_call(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss, out, wgrad_f32=wgrad_f32)
    there = _loss_place(f.device, stream)
    if there is not None:
        with there:
            return fwd_bwd(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss, mode, path, chunk_cells, blank,
                           out, check, None, loss, wgrad_f32, dropout)
    if dropout is not None:
        return _with_dropout(dropout, f, g, out, lambda f, g: fwd_bwd(
            f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss, mode, path, chunk_cells, blank, out, check,
            None, loss, wgrad_f32))
    dtype = "bf16" if f.dtype == torch.bfloat16 else "f32"
    dims = dims_of(f, g, W_o, dtype, mode, path, chunk_cells, blank, loss, wgrad_f32=wgrad_f32)
    if out is None:
        out = Outputs(f, g, W_f, W_g, W_o, b_o, dims)
    rc = lib().frnnt_fwd_bwd(ctypes.byref(dims), _ptr(f), _ptr(g), _ptr(W_f), _ptr(W_g), _ptr(W_o), _ptr(b_o),
                             _ptr(labels), _ptr(T_len), _ptr(U_len), _ptr(grad_loss), _ptr(out.loss),
                             _ptr(out.df), _ptr(out.dg), _ptr(out.dW_f), _ptr(out.dW_g), _ptr(out.dW_o),
                             _ptr(out.db_o), _ptr(out.workspace), out.workspace.numel(), _ptr(out.status),
                             _queue(f.device))
    if rc != OK:
        raise FrnntError(rc, error_string(rc))
    if check:
        bits = int(out.status[0].item())
        if bits:
            raise FrnntStatusError(bits)
    return out.loss, out.grads()


def fwd_bwd_noalloc(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss=None, mode="tiled", path="auto",
                    chunk_cells=0, blank=0, out: Outputs | None = None, check=True, stream=None,
                    loss="marginal", dropout: Dropout | None = None):
    """frnnt_fwd_bwd_noalloc: like fwd_bwd, but the library's fixed scratch
    array replaces the workspace (``out.workspace`` is not used).  Raises
    FrnntError(FRNNT_ERR_WORKSPACE) when these dims need more than
    NOALLOC_MAX_BYTES of scratch."""
    _check_call(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss, out)
    there = _loss_place(f.device, stream)
    if there is not None:
        with there:
            return fwd_bwd_noalloc(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss, mode, path, chunk_cells,
                                   blank, out, check, None, loss, dropout)
    if dropout is not None:
        return _with_dropout(dropout, f, g, out, lambda f, g: fwd_bwd_noalloc(
            f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss, mode, path, chunk_cells, blank, out, check,
            None, loss))
    dtype = "bf16" if f.dtype == torch.bfloat16 else "f32"
    dims = dims_of(f, g, W_o, dtype, mode, path, chunk_cells, blank, loss)
    if out is None:
        out = Outputs(f, g, W_f, W_g, W_o, b_o, dims, with_workspace=False)
    rc = lib().frnnt_fwd_bwd_noalloc(ctypes.byref(dims), _ptr(f), _ptr(g), _ptr(W_f), _ptr(W_g), _ptr(W_o),
                                     _ptr(b_o), _ptr(labels), _ptr(T_len), _ptr(U_len), _ptr(grad_loss),
                                     _ptr(out.loss), _ptr(out.df), _ptr(out.dg), _ptr(out.dW_f), _ptr(out.dW_g),
                                     _ptr(out.dW_o), _ptr(out.db_o), _ptr(out.status),
                                     _queue(f.device))
    if rc != OK:
        msg = error_string(rc)
        if rc == 3:
            msg += f" (these dims need {workspace_size(dims)} bytes; the fixed scratch holds {NOALLOC_MAX_BYTES})"
        raise FrnntError(rc, msg)
    if check:
        bits = int(out.status[0].item())
        if bits:
            raise FrnntStatusError(bits)
    return out.loss, out.grads()


def test_gemm_bf16(A, B, a_mn: bool, b_mn: bool, M: int, N: int, K: int, epi: int = 0, k_splits: int = 1,
                   out=None, stream=None, variant: int = -1, status=None):
    """Test hook: the tensor-core GEMM D = A * B (see include/frnnt_testing.h).
    A is [M][K] (a_mn False) or [K][M]; B is [N][K] (b_mn False) or [K][N]."""
    if out is None:
        out = torch.zeros(M, N, dtype=torch.bfloat16 if epi in (1, 3) else torch.float32, device=A.device)
    if stream is None:
        stream = torch.cuda.current_stream(A.device)
    rc = lib().frnnt_test_gemm_bf16(M, N, K, _ptr(A), int(a_mn), A.stride(0), _ptr(B), int(b_mn), B.stride(0), epi,
                                    k_splits, _ptr(out), out.stride(0), variant, _ptr(status),
                                    ctypes.c_void_p(stream.cuda_stream))
    if rc != OK:
        raise FrnntError(rc, error_string(rc))
    return out


def lose_gemm_loads(n: int) -> int:
    """Test setting (include/frnnt_testing.h): the next n tensor-core GEMM
    launches drop their first K block load, so their bounded wait runs out and
    the status word gets STATUS_TIMEOUT.  Returns the previous count."""
    return int(lib().frnnt_test_lose_gemm_loads(int(n)))


def lose_scan_maps(n: int, round: int = 0, quit: bool = False, tries: int = 200) -> int:
    """Test setting (include/frnnt_testing.h): in the next n recurrence launches
    with clusters of blocks, one block of each withholds its message of a round
    (or gives up after it), so bounded waits run out and the status word gets
    STATUS_TIMEOUT.  Returns the launches that were still to come."""
    return int(lib().frnnt_test_lose_scan_maps(int(n), int(round), int(quit), int(tries)))


def refuse_clusters(on: bool) -> bool:
    """Test setting (include/frnnt_testing.h): the recurrence's requests for
    clusters of blocks fail while it is on.  Returns the previous setting."""
    return bool(lib().frnnt_test_refuse_clusters(int(on)))


def set_joint_variant(variant: int) -> int:
    """Test hook: fused joint kernel variant for later calls (-1 automatic,
    0 one CTA per cell tile, 1 CTA pairs); returns the previous setting."""
    return int(lib().frnnt_test_joint_variant(int(variant)))


def fwd_bwd_pruned(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, bounds, S: int, grad_loss=None, mode="tiled",
                   path="auto", chunk_cells=0, blank=0, out: Outputs | None = None, check=True, stream=None,
                   loss="marginal", wgrad_f32=False, dropout: Dropout | None = None):
    """frnnt_fwd_bwd_pruned: the loss and gradients on the pruned lattice that
    keeps, for frame t of utterance b, the S label positions
    bounds[b,t] <= u < bounds[b,t] + S (bounds: int32 [B, T] on the device)."""
    _check_call(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss, out, bounds=bounds, wgrad_f32=wgrad_f32)
    there = _loss_place(f.device, stream)
    if there is not None:
        with there:
            return fwd_bwd_pruned(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, bounds, S, grad_loss, mode, path,
                                  chunk_cells, blank, out, check, None, loss, wgrad_f32, dropout)
    if dropout is not None:
        return _with_dropout(dropout, f, g, out, lambda f, g: fwd_bwd_pruned(
            f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, bounds, S, grad_loss, mode, path, chunk_cells, blank, out,
            check, None, loss, wgrad_f32))
    dtype = "bf16" if f.dtype == torch.bfloat16 else "f32"
    dims = dims_of(f, g, W_o, dtype, mode, path, chunk_cells, blank, loss, S, wgrad_f32=wgrad_f32)
    if out is None:
        out = Outputs(f, g, W_f, W_g, W_o, b_o, dims)
    rc = lib().frnnt_fwd_bwd_pruned(ctypes.byref(dims), _ptr(f), _ptr(g), _ptr(W_f), _ptr(W_g), _ptr(W_o),
                                    _ptr(b_o), _ptr(labels), _ptr(T_len), _ptr(U_len), _ptr(bounds),
                                    _ptr(grad_loss), _ptr(out.loss), _ptr(out.df), _ptr(out.dg), _ptr(out.dW_f),
                                    _ptr(out.dW_g), _ptr(out.dW_o), _ptr(out.db_o), _ptr(out.workspace),
                                    out.workspace.numel(), _ptr(out.status), _queue(f.device))
    if rc != OK:
        raise FrnntError(rc, error_string(rc))
    if check:
        bits = int(out.status[0].item())
        if bits:
            raise FrnntStatusError(bits)
    return out.loss, out.grads()


def fwd_bwd_tdt(f, g, W_f, W_g, W_o, b_o, W_d, b_d, labels, T_len, U_len, durations, grad_loss=None,
                mode="tiled", chunk_cells=0, blank=0, out: Outputs | None = None, check=True, stream=None,
                wgrad_f32=False, dropout: Dropout | None = None):
    """frnnt_fwd_bwd_tdt: the token-and-duration transducer loss and gradients.

    W_d [n_dur, H] and b_d [n_dur] are the duration head (bf16, like the other
    weights); ``durations`` is the duration set (frame counts, increasing,
    starting 0, 1).  Returns (loss [B] fp32, dict of gradients including dW_d
    and db_d)."""
    _check_call(f, g, W_f, W_g, W_o, b_o, labels, T_len, U_len, grad_loss, out, W_d=W_d, b_d=b_d,
                wgrad_f32=wgrad_f32)
    there = _loss_place(f.device, stream)
    if there is not None:
        with there:
            return fwd_bwd_tdt(f, g, W_f, W_g, W_o, b_o, W_d, b_d, labels, T_len, U_len, durations, grad_loss, mode,
                               chunk_cells, blank, out, check, None, wgrad_f32, dropout)
    if dropout is not None:
        return _with_dropout(dropout, f, g, out, lambda f, g: fwd_bwd_tdt(
            f, g, W_f, W_g, W_o, b_o, W_d, b_d, labels, T_len, U_len, durations, grad_loss, mode, chunk_cells, blank,
            out, check, None, wgrad_f32))
    dtype = "bf16" if f.dtype == torch.bfloat16 else "f32"
    dims = dims_of(f, g, W_o, dtype, mode, "auto", chunk_cells, blank, "marginal", 0, tuple(durations),
                   wgrad_f32=wgrad_f32)
    if out is None:
        out = Outputs(f, g, W_f, W_g, W_o, b_o, dims, W_d=W_d, b_d=b_d)
    rc = lib().frnnt_fwd_bwd_tdt(ctypes.byref(dims), _ptr(f), _ptr(g), _ptr(W_f), _ptr(W_g), _ptr(W_o), _ptr(b_o),
                                 _ptr(W_d), _ptr(b_d), _ptr(labels), _ptr(T_len), _ptr(U_len), _ptr(grad_loss),
                                 _ptr(out.loss), _ptr(out.df), _ptr(out.dg), _ptr(out.dW_f), _ptr(out.dW_g),
                                 _ptr(out.dW_o), _ptr(out.db_o), _ptr(out.dW_d), _ptr(out.db_d),
                                 _ptr(out.workspace), out.workspace.numel(), _ptr(out.status),
                                 _queue(f.device))
    if rc != OK:
        raise FrnntError(rc, error_string(rc))
    if check:
        bits = int(out.status[0].item())
        if bits:
            raise FrnntStatusError(bits)
    return out.loss, out.grads()


# ------------------------------------------------------------------ operators beside the loss (include/frnnt_ops.h)
# These calls can be a few microseconds long on the GPU, so the host side is kept short: each tensor is checked once and
# nothing is built that the call does not need.  Three of PyTorch's own shortcuts are used where this build has them: the
# current stream's handle without a Stream object (0.1 us instead of 2.3), the caching allocator without the dispatcher
# (0.8 us a tensor instead of 1.5 to 2.3), and the current device without the check that CUDA is up (a CUDA tensor is
# at hand).
_TYPES = {torch.float32: F32, torch.bfloat16: BF16}
_I32, _F32T = torch.int32, torch.float32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
try:
    from torch._C._dynamo.guards import _empty_strided_cuda as _new   # (shape, strides, dtype), on the current device
except ImportError:
    def _new(shape, strides, dtype):
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


def _float_type(name, t):
    dt = _TYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be float32 or bfloat16, not {t.dtype}")
    return dt


def _expect(name, t, shape, dtype, dev, dense=True):
    """Refuses a tensor of another shape, type, device or (``dense``) layout than the call needs."""
    if t.shape == shape and t.dtype is dtype and t.device == dev and (not dense or t.is_contiguous()):
        return
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the call's tensors on {dev}")
    raise ValueError(f"{name} must be contiguous")


def _rows(name, t):
    """Elements from one row of a [N, C] tensor to the next (its columns must be adjacent)."""
    N, C = t.shape
    sn, sc = t.stride()
    if C > 1 and sc != 1:
        raise ValueError(f"the columns of {name} must be adjacent (stride 1)")
    return sn if N > 1 else max(C, sn)


def _steps(name, t):
    """(sequence stride, step stride) of a [B, T, D] tensor (its channels must be adjacent)."""
    sb, st, sd = t.stride()
    if sd != 1 and t.shape[2] > 1:
        raise ValueError(f"the channels of {name} must be adjacent (stride 1)")
    return sb, st


def _elsewhere(dev, stream):
    """None where a call on ``dev`` is to be queued on the current stream of the
    current device; otherwise a context that makes it so, for the call's
    outputs (which then belong to that device and stream) and its launch."""
    if dev.type != "cuda":
        raise ValueError("the library computes on the GPU: pass CUDA tensors")
    if stream is None:
        return None if _current_device() == dev.index else torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the call's tensors on {dev}")
    return torch.cuda.stream(stream)


def _queue(dev):
    """The current stream's handle on the current device."""
    return _raw_stream(dev.index) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream


def _status(check, dev):
    return torch.zeros(1, dtype=torch.int32, device=dev) if check else None


def _finish(rc, status):
    if rc != OK:
        raise FrnntError(rc, error_string(rc))
    if status is not None:
        bits = int(status.item())
        if bits:
            raise FrnntStatusError(bits)


def _at(t):
    return None if t is None else t.data_ptr()


class LogProbs:
    """Outputs of token_logprobs: logp [N, K], entropy [N], lse [N], top_logp
    [N, top] (fp32) and top_ids [N, top] (int32); logp is None without tokens,
    the last two are None with top = 0.  lse_rest [N] is what rounding took from
    lse, for the backward call."""
    __slots__ = ("logp", "entropy", "lse", "lse_rest", "top_logp", "top_ids")

    def __init__(self, N, K, top, device):
        def new(dtype, *shape):
            return torch.empty(shape, dtype=dtype, device=device)
        self.logp = new(_F32T, N, K) if K else None
        self.entropy, self.lse, self.lse_rest = (new(_F32T, N) for _ in range(3))
        self.top_logp = new(_F32T, N, top) if top else None
        self.top_ids = new(_I32, N, top) if top else None

    @classmethod
    def _here(cls, N, K, top):
        """The same on the current device."""
        r = cls.__new__(cls)
        r.logp = _new((N, K), (K, 1), _F32T) if K else None
        r.entropy = _new((N,), (1,), _F32T)
        r.lse = _new((N,), (1,), _F32T)
        r.lse_rest = _new((N,), (1,), _F32T)
        if top:
            r.top_logp = _new((N, top), (top, 1), _F32T)
            r.top_ids = _new((N, top), (top, 1), _I32)
        else:
            r.top_logp = r.top_ids = None
        return r


def _check_logprobs(logits, tokens, top):
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError("logits must be [N, V]")
    dt = _TYPES.get(logits.dtype)
    if dt is None:
        _float_type("logits", logits)
    N, V = shape
    K = 0
    if tokens is not None:
        shape = tokens.shape
        if len(shape) != 2:
            raise ValueError("tokens must be [N, K]")
        K = shape[1]
        if shape[0] != N or tokens.dtype is not _I32 or tokens.device != logits.device or not tokens.is_contiguous():
            _expect("tokens", tokens, (N, K), _I32, logits.device)
    if top < 0 or top > V or top > MAX_TOP or K > MAX_TOKENS:
        raise ValueError(f"at most {MAX_TOKENS} tokens and min(V, {MAX_TOP}) alternatives per row")
    sn, sc = logits.stride()
    if sc != 1 and V > 1:
        raise ValueError("the columns of logits must be adjacent (stride 1)")
    return dt, N, V, K, sn if N > 1 else max(V, sn)


def _check_result(fwd, N, K, top, dev):
    f32 = torch.float32
    for name, t, n, dt in (("logp", fwd.logp, K, f32), ("top_logp", fwd.top_logp, top, f32),
                           ("top_ids", fwd.top_ids, top, torch.int32)):
        if t is not None:
            _expect(name, t, (N, n), dt, dev)
        elif n:
            raise ValueError(f"the result has no {name}")
    _expect("entropy", fwd.entropy, (N,), f32, dev)
    _expect("lse", fwd.lse, (N,), f32, dev)
    _expect("lse_rest", fwd.lse_rest, (N,), f32, dev)


def token_logprobs(logits, tokens=None, top=0, out: LogProbs | None = None, check=True, stream=None) -> LogProbs:
    """frnnt_token_logprobs: of each row of logits [N, V] (float32 or bfloat16;
    rows may be strided), the log-probabilities of its given tokens (int32
    [N, K]; NO_TOKEN = none), its entropy and log-sum-exp, and its ``top``
    largest log-probabilities with their columns (ties: lowest column first).
    -inf logits have probability 0.  ``out``: an earlier call's result, written
    again.  With ``check`` the device status is read back (which synchronises)
    and tokens outside [0, V) raise FrnntStatusError."""
    dt, N, V, K, ld = _check_logprobs(logits, tokens, top)
    dev = logits.device
    if out is not None:
        _check_result(out, N, K, top, dev)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return token_logprobs(logits, tokens, top, out, check)
    if out is None:
        out = LogProbs._here(N, K, top)
    status = _status(check and K > 0, dev)
    rc = lib().frnnt_token_logprobs(LogprobDims(N, V, K, top, dt, ld, V, out.lse_rest.data_ptr()),
                                    logits.data_ptr(), _at(tokens), _at(out.logp), out.entropy.data_ptr(),
                                    out.lse.data_ptr(), _at(out.top_logp), _at(out.top_ids), _at(status), _queue(dev))
    if rc or status is not None:
        _finish(rc, status)
    return out


def token_logprobs_bwd(logits, tokens, fwd: LogProbs, dlogp=None, dentropy=None, dtop=None, out=None, check=True,
                       stream=None):
    """frnnt_token_logprobs_bwd: the gradient of sum(logp * dlogp) +
    sum(entropy * dentropy) + sum(top_logp * dtop) for the logits, in their
    type.  ``fwd`` is the forward call's result on the same logits and tokens;
    each of dlogp [N, K], dentropy [N] and dtop [N, top] (fp32) may be None.
    ``out`` [N, V] may be ``logits`` itself (written in place)."""
    top = 0 if fwd.top_ids is None else fwd.top_ids.shape[-1]
    dt, N, V, K, ld = _check_logprobs(logits, tokens, top)
    dev = logits.device
    _check_result(fwd, N, K, top, dev)
    if dlogp is not None:
        _expect("dlogp", dlogp, (N, K), torch.float32, dev)
    if dentropy is not None:
        _expect("dentropy", dentropy, (N,), torch.float32, dev)
    if dtop is not None:
        _expect("dtop", dtop, (N, top), torch.float32, dev)
    if out is not None:
        _expect("out", out, (N, V), logits.dtype, dev, dense=False)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return token_logprobs_bwd(logits, tokens, fwd, dlogp, dentropy, dtop, out, check)
    if out is None:
        out = _new((N, V), (V, 1), logits.dtype)
        ldd = V
    else:
        ldd = _rows("out", out)
    status = _status(check, dev)
    rc = lib().frnnt_token_logprobs_bwd(LogprobDims(N, V, K, top, dt, ld, ldd, fwd.lse_rest.data_ptr()),
                                        logits.data_ptr(), _at(tokens), fwd.lse.data_ptr(), fwd.entropy.data_ptr(),
                                        _at(fwd.top_ids), _at(dlogp), _at(dentropy), _at(dtop), out.data_ptr(),
                                        _at(status), _queue(dev))
    _finish(rc, status)
    return out


class Recurrence:
    """Outputs of recurrence: h [B, T, D], h_last [B, D] (fp32) and, for the
    backward call, the states saved every SCAN_CHUNK steps (fp32)."""
    __slots__ = ("h", "h_last", "saved")

    def __init__(self, B, T, D, dtype, device, save=True):
        self.h = torch.empty((B, T, D), dtype=dtype, device=device)
        self.h_last = torch.empty((B, D), dtype=_F32T, device=device)
        self.saved = torch.empty((B, _marks(T), D), dtype=_F32T, device=device) if save else None

    @classmethod
    def _here(cls, B, T, D, dtype, save):
        """The same on the current device."""
        r = cls.__new__(cls)
        r.h = _new((B, T, D), (T * D, D, 1), dtype)
        r.h_last = _new((B, D), (D, 1), _F32T)
        n = _marks(T)
        r.saved = _new((B, n, D), (n * D, D, 1), _F32T) if save else None
        return r


def _marks(T):
    return (T + SCAN_CHUNK - 1) // SCAN_CHUNK


def _check_recurrence(x, gate, lengths):
    if x.dim() != 3:
        raise ValueError("x and gate must be [B, T, D]")
    dt = _float_type("x", x)
    B, T, D = x.shape
    _expect("gate", gate, (B, T, D), x.dtype, x.device, dense=False)
    if lengths is not None:
        _expect("lengths", lengths, (B,), torch.int32, x.device)
    return dt, B, T, D


def recurrence(x, gate, lengths=None, h0=None, save=True, out: Recurrence | None = None, check=True,
               stream=None) -> Recurrence:
    """frnnt_recurrence_fwd: h_t = a_t h_{t-1} + (1 - a_t) x_t with a =
    sigmoid(gate), over x and gate [B, T, D] (float32 or bfloat16; sequences
    and steps may be strided, as the halves of one projection are), from h0
    [B, D] (fp32; zero when None), each sequence to its length (int32 [B]; T
    when None; rows past it come back 0).  ``save`` keeps what recurrence_bwd
    needs.  ``out``: an earlier call's result, written again."""
    dt, B, T, D = _check_recurrence(x, gate, lengths)
    dev = x.device
    if h0 is not None:
        _expect("h0", h0, (B, D), torch.float32, dev)
    if out is not None:
        _expect("out.h", out.h, (B, T, D), x.dtype, dev, dense=False)
        _expect("out.h_last", out.h_last, (B, D), torch.float32, dev)
        if out.saved is not None:
            _expect("out.saved", out.saved, (B, _marks(T), D), torch.float32, dev)
    strides = _steps("x", x) + _steps("gate", gate)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return recurrence(x, gate, lengths, h0, save, out, check)
    if out is None:
        out = Recurrence._here(B, T, D, x.dtype, save)
        strides += (T * D, D)
    else:
        strides += _steps("out.h", out.h)
    status = _status(check, dev)
    rc = lib().frnnt_recurrence_fwd(RecurrenceDims(B, T, D, dt, *strides), x.data_ptr(), gate.data_ptr(),
                                    _at(lengths), _at(h0), out.h.data_ptr(), out.h_last.data_ptr(), _at(out.saved),
                                    _at(status), _queue(dev))
    _finish(rc, status)
    return out


def recurrence_bwd(x, gate, fwd: Recurrence, dh, lengths=None, dh_last=None, out: dict | None = None, check=True,
                   stream=None) -> dict:
    """frnnt_recurrence_bwd: the gradients dx, dgate [B, T, D] (type of x) and
    dh0 [B, D] (fp32) of sum(h * dh) + sum(h_last * dh_last).  ``fwd`` is the
    forward call's result (only its saved states are read) on the same x, gate
    and lengths.  ``out``: a dict with dx, dgate and dh0 to write to (dx and
    dgate may be the halves of one gradient)."""
    dt, B, T, D = _check_recurrence(x, gate, lengths)
    dev = x.device
    if fwd.saved is None:
        raise ValueError("the forward call kept no states (save=False)")
    _expect("fwd.saved", fwd.saved, (B, _marks(T), D), torch.float32, dev)
    _expect("dh", dh, (B, T, D), x.dtype, dev, dense=False)
    if dh_last is not None:
        _expect("dh_last", dh_last, (B, D), torch.float32, dev)
    if out is not None:
        _expect("out dx", out["dx"], (B, T, D), x.dtype, dev, dense=False)
        _expect("out dgate", out["dgate"], (B, T, D), x.dtype, dev, dense=False)
        _expect("out dh0", out["dh0"], (B, D), torch.float32, dev)
    strides = _steps("x", x) + _steps("gate", gate) + (0, 0) + _steps("dh", dh)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return recurrence_bwd(x, gate, fwd, dh, lengths, dh_last, out, check)
    if out is None:
        full = (T * D, D, 1)
        out = dict(dx=_new((B, T, D), full, x.dtype), dgate=_new((B, T, D), full, x.dtype),
                   dh0=_new((B, D), (D, 1), _F32T))
        strides += (T * D, D, T * D, D)
    else:
        strides += _steps("out dx", out["dx"]) + _steps("out dgate", out["dgate"])
    status = _status(check, dev)
    rc = lib().frnnt_recurrence_bwd(RecurrenceDims(B, T, D, dt, *strides), x.data_ptr(), gate.data_ptr(),
                                    _at(lengths), fwd.saved.data_ptr(), dh.data_ptr(), _at(dh_last),
                                    out["dx"].data_ptr(), out["dgate"].data_ptr(), out["dh0"].data_ptr(),
                                    _at(status), _queue(dev))
    _finish(rc, status)
    return out


def recurrence_step(x, gate, state, parent=None, advance=None, out=None, check=True, stream=None):
    """frnnt_recurrence_step: one step of N hypotheses.  Row n of x and gate [N,
    D] continues row parent[n] of state [S, D] (fp32; row n when parent is
    None), or only copies it where advance[n] (bool) is False.  Returns (h [N,
    D] in the type of x, new state [N, D] fp32); ``out``: that pair to write
    to.  The new state may be written over ``state`` when parent is None."""
    if x.dim() != 2 or state.dim() != 2:
        raise ValueError("x and gate must be [N, D] and state [S, D]")
    dt = _float_type("x", x)
    dev = x.device
    N, D = x.shape
    S = state.shape[0]
    _expect("gate", gate, (N, D), x.dtype, dev, dense=False)
    _expect("state", state, (S, D), torch.float32, dev)
    if parent is not None:
        _expect("parent", parent, (N,), torch.int32, dev)
    elif N > S:
        raise ValueError(f"{N} rows need parents among the {S} rows of state")
    if advance is not None:
        _expect("advance", advance, (N,), torch.bool, dev)
    x_sn, gate_sn = _rows("x", x), _rows("gate", gate)
    if out is not None:
        h, new = out
        _expect("out h", h, (N, D), x.dtype, dev)
        _expect("out state", new, (N, D), torch.float32, dev)
        old, at = state.data_ptr(), new.data_ptr()
        if (parent is not None or at != old) and at < old + S * D * 4 and old < at + N * D * 4:
            raise ValueError("the new state overlaps the old one, which other rows still read")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return recurrence_step(x, gate, state, parent, advance, out, check)
    if out is None:
        h = _new((N, D), (D, 1), x.dtype)
        new = _new((N, D), (D, 1), _F32T)
    status = _status(check and parent is not None, dev)
    rc = lib().frnnt_recurrence_step(StepDims(N, S, D, dt, x_sn, gate_sn), x.data_ptr(), gate.data_ptr(),
                                     state.data_ptr(), _at(parent), _at(advance), h.data_ptr(), new.data_ptr(),
                                     _at(status), _queue(dev))
    _finish(rc, status)
    return h, new


def _matrix(name, t):
    """(rows, elements per row, row stride) of a tensor whose elements, in
    row-major order, are rows at one constant distance."""
    if t.is_contiguous():
        n = t.numel()
        return 1, n, n
    C = t.shape[-1]
    if t.stride(-1) == 1 or C == 1:
        if t.dim() == 2:
            return t.shape[0], C, t.stride(0)
        try:
            v = t.view(-1, C)
        except RuntimeError:
            pass
        else:
            return v.shape[0], C, v.stride(0)
    raise ValueError(f"{name} must be contiguous, or rows at a constant distance")


def dropout(x, p, seed, offset=0, out=None, stream=None):
    """frnnt_dropout: x with each element dropped with probability p (0 .. 1)
    and the others scaled by 1 / (1 - p); float32 or bfloat16, any shape.  The
    mask depends on (seed, offset) and the element's row-major index alone, so
    the same call on the gradient is the backward pass.  One call uses
    ceil(numel / 8) counters from ``offset`` on.  ``seed``: an int, or an int64
    CUDA tensor (seed, offset) read on the device, whose second value is added
    to ``offset`` (a captured graph then draws new numbers at each replay).
    ``out`` may be x."""
    dt = _float_type("x", x)
    dev = x.device
    if x.numel() == 0:
        raise ValueError("x has no elements")
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be in [0, 1], not {p}")
    rng, key = None, seed
    if isinstance(seed, torch.Tensor):
        rng, key = seed, 0
        _expect("seed", rng, (2,), torch.int64, dev)
    R, C, x_ld = _matrix("x", x)
    y_ld = C
    if out is not None:
        _expect("out", out, x.shape, x.dtype, dev, dense=False)
        Ry, Cy, y_ld = _matrix("out", out)
        if (R, C) != (Ry, Cy):     # one of the two is contiguous: take the rows of the other
            if R == 1:
                R, C, x_ld = Ry, Cy, Cy
            elif Ry == 1:
                y_ld = C
            else:
                raise ValueError("x and out have rows of different lengths")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return dropout(x, p, seed, offset, out)
    if out is None:
        out = _new(tuple(x.shape), x.stride(), x.dtype) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=dev)
    mask = (1 << 64) - 1
    rc = lib().frnnt_dropout(DropoutDims(R, C, dt, x_ld, y_ld, p, key & mask, offset & mask), x.data_ptr(),
                             out.data_ptr(), _at(rng), _queue(dev))
    _finish(rc, None)
    return out
