"""Rotary positions and the norms of queries and keys (see include/kvp.h).

:class:`Rope` holds a model's frequencies; the functions beside it are the C ABI's calls, with the
checks of shapes, types and devices that need no look at the data.  Gradients are calls of their
own (``kvp_rope`` with ``inverse``, ``kvp_qk_norm_rope_backward``): like the rest of this package
they are not recorded by autograd.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._lib import _DTYPE, _check, _need, load
from .paged import _raw_stream


class _Freqs(ctypes.Structure):
    """kvp_rope_freqs."""
    _fields_ = [("inv_freq", ctypes.POINTER(ctypes.c_double)), ("rotary_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("gain", ctypes.c_double)]


class Rope:
    """The frequencies of a rotation of the first ``rotary_dim`` values of a head.

    inv_freq[i] = theta ** (-2 i / rotary_dim) radians per position for the pairs (i, i + rotary_dim / 2),
    or (2i, 2i + 1) when ``interleaved``; for contexts ``factor`` times longer than the ``original_len``
    a model was trained on, with ``scaling``:

    * ``"linear"``: every frequency divided by the factor (positions interpolated);
    * ``"ntk"``: theta times factor ** (rotary_dim / (rotary_dim - 2)), which leaves the fastest pair as it
      is and divides the slowest by the factor;
    * ``"bands"``: wavelengths above original_len / low divided, those below original_len / high left,
      between them a blend that is linear in the turns within original_len;
    * ``"yarn"``: a ramp over the pairs that turn beta_fast ... beta_slow times within original_len, and
      cosine and sine times 0.1 ln(factor) + 1 (or ``gain``).

    ``inv_freq`` (a sequence of rotary_dim / 2 numbers) gives the frequencies instead.
    """

    def __init__(self, rotary_dim, theta=10000.0, interleaved=False, scaling="none", factor=1.0, original_len=None,
                 low=1.0, high=4.0, beta_fast=32.0, beta_slow=1.0, gain=None, inv_freq=None):
        r = int(rotary_dim)
        if r < 16 or r > 128 or r % 16:
            raise ValueError(f"rotary_dim must be a multiple of 16 in [16, 128], got {rotary_dim}")
        if scaling not in ("none", "linear", "ntk", "bands", "yarn"):
            raise ValueError(f"unknown scaling {scaling!r}")
        if scaling == "none":
            factor = 1.0
        if not (factor > 0 and math.isfinite(factor)):
            raise ValueError(f"factor must be positive and finite, got {factor}")
        if scaling in ("bands", "yarn") and (original_len is None or original_len < 1):
            raise ValueError(f"scaling {scaling!r} needs original_len >= 1")
        if inv_freq is None:
            if not (theta > 1 and math.isfinite(theta)):
                raise ValueError(f"theta must be above 1 and finite, got {theta}")
            inv_freq = self._scaled(r, theta, scaling, factor, original_len, low, high, beta_fast, beta_slow)
        elif scaling != "none":
            raise ValueError("inv_freq is given: it takes no scaling")
        inv_freq = [float(f) for f in inv_freq]
        if len(inv_freq) != r // 2:
            raise ValueError(f"inv_freq must hold {r // 2} numbers, got {len(inv_freq)}")
        if not all(0 <= f <= 1e6 for f in inv_freq):
            raise ValueError("inv_freq must lie in [0, 1e6]")
        if gain is None:
            gain = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0
        if not math.isfinite(gain):
            raise ValueError("gain must be finite")
        self.rotary_dim, self.interleaved, self.gain, self.inv_freq = r, bool(interleaved), float(gain), tuple(inv_freq)
        self._array = (ctypes.c_double * (r // 2))(*inv_freq)
        self._desc = _Freqs(self._array, r, int(self.interleaved), self.gain)
        self._ref = ctypes.byref(self._desc)

    @staticmethod
    def _scaled(r, theta, scaling, factor, n, low, high, beta_fast, beta_slow):
        if scaling == "ntk":
            if r <= 2:
                raise ValueError("ntk scaling needs more than one pair")
            theta *= factor ** (r / (r - 2))
        inv = [theta ** (-2 * i / r) for i in range(r // 2)]
        if scaling == "linear":
            return [f / factor for f in inv]
        if scaling == "bands":
            if not high > low:
                raise ValueError("bands need high > low")
            keep = [min(max((n * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for f in inv]
            return [(1 - s) * f / factor + s * f for f, s in zip(inv, keep)]
        if scaling == "yarn":
            if not beta_fast > beta_slow > 0:
                raise ValueError("yarn needs beta_fast > beta_slow > 0")

            def pair(turns):             # the (fractional) pair that turns so often within n positions
                return r * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(theta))
            lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), r - 1)
            ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(r // 2)]
            return [f / factor * t + f * (1 - t) for f, t in zip(inv, ramp)]
        return inv


def _elsewhere(index, stream):
    return stream is not None or torch.cuda.current_device() != index


def _there(index, stream):
    """The call's device and stream made the current ones, so that its temporaries belong to them."""
    if stream is None:
        return torch.cuda.device(index)
    if stream.device != torch.device("cuda", index):
        raise ValueError(f"stream must be on cuda:{index}, got {stream.device}")
    return torch.cuda.stream(stream)


_Strides = ctypes.c_int64 * 3


def _rows(t, name, like=None, heads=None):
    """[B, H, S, D] or [H, S, D] with a contiguous last axis, of the same device, type and sizes as ``like`` (but for
    ``heads``): (pointer, strides or None, (device index, dtype, B, H, S, D)).  A small call is its checks, so each
    attribute is asked for once."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index, dtype, shape = t.get_device(), t.dtype, t.shape
    if index < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    n = len(shape)
    if n == 4:
        B, H, S, D = shape
    elif n == 3:
        B = 1
        H, S, D = shape
    else:
        raise ValueError(f"{name} must be [B, H, S, D] or [H, S, D]")
    this = (index, dtype, B, H, S, D)
    if like is not None:
        want = like if heads is None else like[:3] + (heads,) + like[4:]
        if this != want:
            if index != want[0]:
                raise ValueError(f"{name} must be on cuda:{want[0]}, got {t.device}")
            if dtype != want[1]:
                raise ValueError(f"{name} must be {want[1]}, got {dtype}")
            raise ValueError(f"{name} must have shape {want[2:]}, got {this[2:]}")
    if t.is_contiguous():
        return t.data_ptr(), None, this
    strides = t.stride()
    if strides[-1] != 1:
        raise ValueError(f"{name}: the head_dim axis must be contiguous")
    return t.data_ptr(), _Strides(*strides[:3]) if n == 4 else _Strides(0, *strides[:2]), this


def _result(out, name, x, like):
    """The tensor to return, like x: `out`, or a new dense one; (tensor, pointer, strides)."""
    if out is None:
        out = torch.empty(x.shape, dtype=like[1], device=x.device)
        return out, out.data_ptr(), None
    ptr, strides, _ = _rows(out, name, like)
    return out, ptr, strides


def _positions(positions, like):
    """int32 [S] or [B, S] (rows of consecutive positions in memory): (pointer, stride)."""
    if positions is None:
        return None, 0
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch.Tensor")
    B, S = like[2], like[4]
    if positions.get_device() != like[0]:
        raise ValueError(f"positions must be on cuda:{like[0]}, got {positions.device}")
    if positions.dtype != torch.int32:
        raise ValueError(f"positions must be torch.int32, got {positions.dtype}")
    shape = positions.shape
    if shape != (B, S) and shape != (S,):
        raise ValueError(f"positions must have shape ({S},) or ({B}, {S}), got {tuple(shape)}")
    strides = positions.stride()
    if S > 1 and strides[-1] != 1:
        raise ValueError("positions must be contiguous along the tokens")
    return positions.data_ptr(), strides[0] if len(strides) == 2 and B > 1 else 0


def _start(start):
    """(An int that is passed to C as 32 bits would lose the others.)"""
    start = int(start)
    if not -1 << 31 <= start < 1 << 31:
        raise ValueError(f"start must fit 32 bits, got {start}")
    return start


def _rope_ref(rope):
    if rope is None:
        return None
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    return rope._ref


def _code(dtype):
    code = _DTYPE.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    return code


def kvp_rope(x, rope, positions=None, start=0, inverse=False, out=None, stream=None):
    """Rotate x [B, H, S, D] (or [H, S, D]; strided views are read in place) by the positions of its tokens:
    int32 [S] or [B, S], or start, start + 1, ...  ``inverse`` turns back (the rotation's gradient; keys that are
    moved back to other positions take a ``rope`` of gain 1: they have the rotation's already).  ``out`` may
    be x itself; by default a new dense tensor."""
    x_ptr, xs, like = _rows(x, "x")
    index, dtype, B, H, S, D = like
    if _elsewhere(index, stream):
        with _there(index, stream):
            return kvp_rope(x, rope, positions, start, inverse, out)
    if rope is None:
        raise TypeError("rope must be a Rope")
    dtype = _code(dtype)
    out, out_ptr, os = _result(out, "out", x, like)
    pos, ps = _positions(positions, like)
    rc = load().kvp_rope(x_ptr, out_ptr, dtype, B, H, S, D, xs, os, _rope_ref(rope), pos, ps, _start(start),
                         int(bool(inverse)), _raw_stream(index))
    if rc:
        _check("kvp_rope", rc)
    return out


def _weight(w, name, like):
    """[D] of the tensors' type or float32: (pointer, dtype)."""
    if w is None:
        return None, None
    if not isinstance(w, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index, dtype = w.get_device(), w.dtype
    if index < 0 or not w.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if w.shape != like[5:]:
        raise ValueError(f"{name} must have shape {like[5:]}, got {tuple(w.shape)}")
    if index != like[0]:
        raise ValueError(f"{name} must be on cuda:{like[0]}, got {w.device}")
    if dtype != like[1] and dtype != torch.float32:
        raise ValueError(f"{name} must be {like[1]} or torch.float32, got {dtype}")
    return w.data_ptr(), dtype


def _weights(q_weight, k_weight, like):
    q, q_dtype = _weight(q_weight, "q_weight", like)
    k, k_dtype = _weight(k_weight, "k_weight", like)
    if q_dtype is not None and k_dtype is not None and q_dtype != k_dtype:
        raise ValueError("q_weight and k_weight must have the same dtype")
    return q, k, _DTYPE[q_dtype or k_dtype or like[1]]


def _heads(k):
    return k.shape[-3] if isinstance(k, torch.Tensor) and k.dim() >= 3 else 0


def kvp_qk_norm_rope(q, k, q_weight=None, k_weight=None, eps=1e-6, rope=None, positions=None, start=0, q_out=None,
                     k_out=None, stream=None):
    """Norms of every head of q [B, H_q, S, D] and k [B, H_kv, S, D] (or without B; strided views are read in
    place) over its D values, times the weights [D] (of q's dtype or float32; None: ones), rotated as by
    :func:`kvp_rope` (rope None: not rotated) -> (q_out, k_out).  The outputs may be q and k themselves."""
    q_ptr, qs, like = _rows(q, "q")
    index, dtype, B, Hq, S, D = like
    if _elsewhere(index, stream):
        with _there(index, stream):
            return kvp_qk_norm_rope(q, k, q_weight, k_weight, eps, rope, positions, start, q_out, k_out)
    dtype = _code(dtype)
    k_ptr, ks, k_like = _rows(k, "k", like, _heads(k))
    q_out, qo_ptr, qos = _result(q_out, "q_out", q, like)
    k_out, ko_ptr, kos = _result(k_out, "k_out", k, k_like)
    pos, ps = _positions(positions, like)
    qw, kw, wd = _weights(q_weight, k_weight, like)
    rc = load().kvp_qk_norm_rope(q_ptr, k_ptr, qo_ptr, ko_ptr, dtype, B, Hq, k_like[3], S, D, qs, ks, qos, kos, qw, kw, wd,
                                 float(eps), _rope_ref(rope), pos, ps, _start(start), _raw_stream(index))
    if rc:
        _check("kvp_qk_norm_rope", rc)
    return q_out, k_out


@functools.lru_cache(maxsize=256)
def _backward_bytes(index, *sizes):
    """(The sizes alone decide, on a device: the current one.)"""
    return int(load().kvp_qk_norm_rope_backward_workspace_size(*sizes))


def kvp_qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight=None, k_weight=None, eps=1e-6, rope=None, positions=None,
                              start=0, dq=None, dk=None, workspace=None, stream=None):
    """Gradients of :func:`kvp_qk_norm_rope` from those of its outputs and its inputs ->
    (dq, dk, dq_weight, dk_weight), the last two float32 [D] (of weights that are None as of ones).
    dq may be dq_out or q itself, dk likewise."""
    q_ptr, qs, like = _rows(q, "q")
    index, dtype, B, Hq, S, D = like
    if _elsewhere(index, stream):
        with _there(index, stream):
            return kvp_qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, eps, rope, positions, start, dq,
                                             dk, workspace)
    dtype = _code(dtype)
    k_ptr, ks, k_like = _rows(k, "k", like, _heads(k))
    gq_ptr, gqs, _ = _rows(dq_out, "dq_out", like)
    gk_ptr, gks, _ = _rows(dk_out, "dk_out", k_like)
    dq, dq_ptr, dqs = _result(dq, "dq", q, like)
    dk, dk_ptr, dks = _result(dk, "dk", k, k_like)
    pos, ps = _positions(positions, like)
    qw, kw, wd = _weights(q_weight, k_weight, like)
    device = q.device
    dwq, dwk = (torch.empty(D, dtype=torch.float32, device=device) for _ in range(2))
    if workspace is None:
        workspace = torch.empty(_backward_bytes(index, dtype, B, Hq, k_like[3], S, D), dtype=torch.uint8, device=device)
    else:
        _need(workspace, "workspace", torch.uint8)
        if workspace.device != device:
            raise ValueError(f"workspace must be on {device}, got {workspace.device}")
    rc = load().kvp_qk_norm_rope_backward(gq_ptr, gk_ptr, q_ptr, k_ptr, dq_ptr, dk_ptr, dwq.data_ptr(), dwk.data_ptr(), dtype,
                                          B, Hq, k_like[3], S, D, gqs, gks, qs, ks, dqs, dks, qw, kw, wd, float(eps),
                                          _rope_ref(rope), pos, ps, _start(start), workspace.data_ptr(), workspace.numel(),
                                          _raw_stream(index))
    if rc:
        _check("kvp_qk_norm_rope_backward", rc)
    return dq, dk, dwq, dwk
