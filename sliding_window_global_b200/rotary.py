"""ctypes binding of the rotation and head norm (swa_rotary_forward / _backward).

Argument marshalling only, as in ``swa.py``: the arithmetic runs in the library's CUDA
kernels, and a call on anything but CUDA tensors raises.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional

import torch

from .swa import SwaError, _dtype_code, load_library

P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class Rotation(ctypes.Structure):
    """swa_rotation of include/swa.h."""
    _fields_ = [("rotary_dim", I), ("interleaved", I), ("freq", P), ("amplitude", F)]


class HeadNorm(ctypes.Structure):
    """swa_head_norm of include/swa.h."""
    _fields_ = [("norm", I), ("eps", F), ("q_weight", P), ("k_weight", P), ("weight_dtype", I)]


class RotaryArgs(ctypes.Structure):
    """swa_rotary_args of include/swa.h (each stride array as its elements)."""
    _fields_ = [
        ("batch", I), ("seq_len", I), ("num_q_heads", I), ("num_kv_heads", I), ("head_dim", I), ("dtype", I),
        ("q", P), ("k", P),
        ("q_stride0", I64), ("q_stride1", I64), ("q_stride2", I64),
        ("k_stride0", I64), ("k_stride1", I64), ("k_stride2", I64),
        ("positions", P), ("start", I), ("q_out", P), ("k_out", P),
        ("q_out_stride0", I64), ("q_out_stride1", I64), ("q_out_stride2", I64),
        ("k_out_stride0", I64), ("k_out_stride1", I64), ("k_out_stride2", I64),
        ("rotation", Rotation), ("head_norm", HeadNorm),
    ]


class RotaryBackwardArgs(ctypes.Structure):
    """swa_rotary_backward_args of include/swa.h (each stride array as its elements)."""
    _fields_ = [
        ("batch", I), ("seq_len", I), ("num_q_heads", I), ("num_kv_heads", I), ("head_dim", I),
        ("dtype", I), ("grad_dtype", I), ("out_dtype", I), ("q", P), ("k", P),
        ("q_stride0", I64), ("q_stride1", I64), ("q_stride2", I64),
        ("k_stride0", I64), ("k_stride1", I64), ("k_stride2", I64),
        ("positions", P), ("start", I), ("dq_out", P), ("dk_out", P),
        ("dq_out_stride0", I64), ("dq_out_stride1", I64), ("dq_out_stride2", I64),
        ("dk_out_stride0", I64), ("dk_out_stride1", I64), ("dk_out_stride2", I64),
        ("dq", P), ("dk", P),
        ("dq_stride0", I64), ("dq_stride1", I64), ("dq_stride2", I64),
        ("dk_stride0", I64), ("dk_stride1", I64), ("dk_stride2", I64),
        ("dq_weight", P), ("dk_weight", P), ("rotation", Rotation), ("head_norm", HeadNorm),
        ("workspace", P), ("workspace_bytes", ctypes.c_size_t),
    ]


# A call of a few microseconds on the GPU is bound by what the host does for it, so the
# paths below take the cheapest spelling of each step: argument structs packed in one go,
# outputs by empty_like, the stream's handle without a Stream object, and a device or stream
# context only where it changes something.
_raw_stream = torch._C._cuda_getCurrentRawStream


def packer(cls):
    """A function that packs the (flattened) field values of a ctypes structure into its
    bytes; pointers are addresses, 0 for NULL."""
    codes = {I: "i", I64: "q", P: "Q", F: "f", ctypes.c_size_t: "Q"}

    def layout(c):
        fmt, at = "", 0
        for name, kind in c._fields_:
            offset = getattr(c, name).offset
            fmt += "x" * (offset - at)
            fmt += layout(kind) if issubclass(kind, ctypes.Structure) else codes[kind]
            at = offset + ctypes.sizeof(kind)
        return fmt + "x" * (ctypes.sizeof(c) - at)

    s = struct.Struct("=" + layout(cls))
    assert s.size == ctypes.sizeof(cls)
    return s.pack


_pack_forward, _pack_backward = packer(RotaryArgs), packer(RotaryBackwardArgs)
NO_STRIDES = (0, 0, 0)
NO_ROTATION = (0, 0, 0, 1.0)               # fields of Rotation, of HeadNorm
_NO_NORM = (0, 0.0, 0, 0, 0)


def elsewhere(t: torch.Tensor, name: str, stream):
    """The context a call on ``t`` must enter first (None: it can run as things are): its
    device current, and ``stream`` the one that outputs and workspaces are allocated for."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
        return torch.cuda.stream(stream)
    if t.get_device() != torch.cuda.current_device():
        return torch.cuda.device(t.device)
    return None


def current_stream(t: torch.Tensor) -> int:
    return _raw_stream(t.get_device())


def check_rows(t: torch.Tensor, name: str, device, dims: int, dtype=None):
    """A tensor of head rows: on ``device``, ``dims`` axes, the last one dense.  Returns its
    strides."""
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != dims:
        raise ValueError(f"{name} needs {dims} axes, got {t.dim()}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    strides = t.stride()
    if strides[-1] != 1 and t.numel() > 0:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return strides


def check_index(t: Optional[torch.Tensor], name: str, device, shape):
    """An int32 tensor of the given shape (or None); returns its address (or 0)."""
    if t is None:
        return 0
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def head_norm(norm_eps, q_weight, k_weight, head_dim: int, device):
    """Fields of swa_head_norm (norm_eps None: no norm)."""
    if norm_eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("norm weights need norm_eps")
        return _NO_NORM
    code, ptrs = 0, []
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            ptrs.append(0)
            continue
        check_rows(w, name, device, 1)
        if w.shape[0] != head_dim:
            raise ValueError(f"{name} must have {head_dim} elements, got {w.shape[0]}")
        ptrs.append(w.data_ptr())
        code = _dtype_code(w.dtype)
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise TypeError("q_weight and k_weight must have one dtype")
    return 1, norm_eps, ptrs[0], ptrs[1], code


def check_fp32(x: float, name: str):
    """A number the library takes as fp32 and for which 0 means something of its own: refused
    where fp32 would round it to 0 or to infinity."""
    if x and math.isfinite(x) and ctypes.c_float(x).value in (0.0, math.inf, -math.inf):
        raise ValueError(f"{name} is outside the range of fp32: {x}")


def check_start(start: int):
    if not -2 ** 31 <= start < 2 ** 31:
        raise ValueError(f"start must be an int32, got {start}")


def rotary_frequencies(rotary_dim: int, *, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original_length: int = 4096, low_turns: float = 1.0, high_turns: float = 32.0):
    """Radians a position for each of the ``rotary_dim / 2`` pairs (fp64, on the host), and
    the amplitude: ``freq[j] = base ** (-2 j / rotary_dim)``, stretched for contexts
    ``factor`` times the trained length:

    - ``"linear"``: every frequency divided by the factor (positions interpolated);
    - ``"ntk"``: the base grows by ``factor ** (rotary_dim / (rotary_dim - 2))``, so that the
      slowest pair is interpolated and the fastest kept;
    - ``"yarn"``: pairs that turn more than ``high_turns`` times over ``original_length`` are
      kept, those below ``low_turns`` interpolated, a linear ramp between, and the rotated
      vectors scaled by ``0.1 ln(factor) + 1``."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if not factor > 0.0 or not base > 0.0:
        raise ValueError("base and factor must be positive")
    j = torch.arange(rotary_dim // 2, dtype=torch.float64)
    if scaling == "ntk":
        if rotary_dim < 4:
            raise ValueError("ntk scaling needs a rotary_dim of 4 or more")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = base ** (-2.0 * j / rotary_dim)
    if scaling in ("none", "ntk"):
        return freq, 1.0
    if scaling == "linear":
        return freq / factor, 1.0
    if scaling == "yarn":
        turns = original_length * freq / (2.0 * math.pi)
        keep = ((turns - low_turns) / (high_turns - low_turns)).clamp(0.0, 1.0)
        return freq * keep + freq / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    raise ValueError(f"unknown scaling {scaling!r}; use none, linear, ntk or yarn")


def _make(head_dim, options):
    return Rotary(head_dim, **options)


class Rotary:
    """Rotation of query and key heads by their positions, with an optional RMS norm of
    every head before it, and its gradients.

    ``rotary_dim`` leading elements of a head rotate (all by default), in pairs
    ``(2j, 2j + 1)`` (``interleaved``) or ``(j, j + rotary_dim / 2)``; ``frequencies`` gives
    the radians a position of each pair (``rotary_frequencies`` makes them; base 10000
    without scaling by default), ``amplitude`` scales the rotated elements."""

    def __init__(self, head_dim: int, *, rotary_dim: Optional[int] = None, interleaved: bool = True,
                 frequencies: Optional[torch.Tensor] = None, amplitude: float = 1.0):
        self._lib = load_library()
        self.head_dim = int(head_dim)
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        self.interleaved = bool(interleaved)
        self.amplitude = float(amplitude)
        if head_dim not in (64, 128) or self.rotary_dim % 16 or not 0 <= self.rotary_dim <= self.head_dim:
            raise ValueError("head_dim must be 64 or 128 and rotary_dim a multiple of 16 up to it, "
                             f"got {head_dim} and {self.rotary_dim}")
        if not math.isfinite(self.amplitude) or self.amplitude == 0.0:
            raise ValueError("amplitude must be finite and not zero")
        check_fp32(self.amplitude, "amplitude")
        if frequencies is None:
            frequencies = rotary_frequencies(self.rotary_dim)[0] if self.rotary_dim else torch.empty(0)
        freq = frequencies.detach().to("cpu", torch.float64).reshape(-1).tolist()
        if len(freq) != self.rotary_dim // 2 or not all(math.isfinite(f) for f in freq):
            raise ValueError(f"frequencies needs {self.rotary_dim // 2} finite values")
        self._freq = (ctypes.c_double * max(1, len(freq)))(*freq)
        self.fields = (self.rotary_dim, int(self.interleaved), ctypes.addressof(self._freq), self.amplitude)

    def __reduce__(self):
        # a copy has its own frequencies, and the library belongs to the process
        freq = torch.tensor(self._freq[:self.rotary_dim // 2], dtype=torch.float64)
        return _make, (self.head_dim, dict(rotary_dim=self.rotary_dim, interleaved=self.interleaved, frequencies=freq,
                                           amplitude=self.amplitude))

    def forward(self, q: torch.Tensor, k: Optional[torch.Tensor] = None, *, positions: Optional[torch.Tensor] = None,
                start: int = 0, norm_eps: Optional[float] = None, q_weight: Optional[torch.Tensor] = None,
                k_weight: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                k_out: Optional[torch.Tensor] = None, stream=None):
        """Rotated q [B, Hq, n, D] and k [B, Hkv, n, D] (any strides with a dense last axis, so
        a slice of a projection's output as it lies); ``positions`` int32 [B, n], or ``start``,
        ``start + 1``, ... in every batch.  ``norm_eps``: norm every head first, times the
        weights [D].  Outputs are contiguous unless given; an output may be its input.
        Returns ``(q_out, k_out)``."""
        ctx = elsewhere(q, "q", stream)
        if ctx is None:
            return self._forward(q, k, positions, start, norm_eps, q_weight, k_weight, q_out, k_out)
        with ctx:
            return self._forward(q, k, positions, start, norm_eps, q_weight, k_weight, q_out, k_out)

    def _forward(self, q, k, positions, start, norm_eps, q_weight, k_weight, q_out, k_out):
        check_start(start)
        device, dtype = q.device, q.dtype
        code = _dtype_code(dtype)
        qs = check_rows(q, "q", device, 4)
        B, Hq, n, D = q.shape
        if D != self.head_dim:
            raise ValueError(f"q has head_dim {D}, expected {self.head_dim}")
        Hkv, ks = 0, NO_STRIDES
        if k is not None:
            ks = check_rows(k, "k", device, 4, dtype)
            Bk, Hkv, nk, Dk = k.shape
            if Bk != B or nk != n or Dk != D:
                raise ValueError(f"k must be [{B}, heads, {n}, {D}], got {tuple(k.shape)}")
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            os = (Hq * n * D, n * D, D)
        else:
            os = self._check_out(q_out, "q_out", q)
        kos, k_ptr, ko_ptr = NO_STRIDES, 0, 0
        if k is None:
            k_out = None
        else:
            if k_out is None:
                k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
                kos = (Hkv * n * D, n * D, D)
            else:
                kos = self._check_out(k_out, "k_out", k)
            k_ptr, ko_ptr = k.data_ptr(), k_out.data_ptr()
        a = _pack_forward(
            B, n, Hq, Hkv, D, code, q.data_ptr(), k_ptr, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2],
            check_index(positions, "positions", device, (B, n)), start, q_out.data_ptr(), ko_ptr,
            os[0], os[1], os[2], kos[0], kos[1], kos[2], *self.fields,
            *head_norm(norm_eps, q_weight, k_weight, D, device))
        st = self._lib.swa_rotary_forward(a, current_stream(q))
        if st != 0:
            raise SwaError(st, "swa_rotary_forward")
        return q_out, k_out

    def backward(self, dq_out: torch.Tensor, dk_out: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                 k: Optional[torch.Tensor] = None, *, positions: Optional[torch.Tensor] = None, start: int = 0,
                 norm_eps: Optional[float] = None, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, dq: Optional[torch.Tensor] = None,
                 dk: Optional[torch.Tensor] = None, stream=None):
        """Gradients for the upstream ``dq_out``, ``dk_out`` (as ``Plan.backward`` gives them, or
        bf16).  ``q``, ``k`` are the forward's inputs, required with a norm; they set the
        gradients' dtype and layout (without them, the upstream's).  Returns ``(dq, dk)``, and
        with a norm ``(dq, dk, dq_weight, dk_weight)`` (fp32 [D]; None without that weight)."""
        ctx = elsewhere(dq_out, "dq_out", stream)
        if ctx is None:
            return self._backward(dq_out, dk_out, q, k, positions, start, norm_eps, q_weight, k_weight, dq, dk)
        with ctx:
            return self._backward(dq_out, dk_out, q, k, positions, start, norm_eps, q_weight, k_weight, dq, dk)

    def _backward(self, dq_out, dk_out, q, k, positions, start, norm_eps, q_weight, k_weight, dq, dk):
        check_start(start)
        device = dq_out.device
        gs = check_rows(dq_out, "dq_out", device, 4)
        B, Hq, n, D = dq_out.shape
        if D != self.head_dim:
            raise ValueError(f"dq_out has head_dim {D}, expected {self.head_dim}")
        Hkv, gks = 0, NO_STRIDES
        if dk_out is not None:
            gks = check_rows(dk_out, "dk_out", device, 4, dq_out.dtype)
            Bk, Hkv, nk, Dk = dk_out.shape
            if Bk != B or nk != n or Dk != D:
                raise ValueError(f"dk_out must be [{B}, heads, {n}, {D}], got {tuple(dk_out.shape)}")
        if norm_eps is not None and (q is None or (k is None and Hkv > 0)):
            raise ValueError("the norm's gradient needs q and k")
        qs = ks = NO_STRIDES
        if q is not None:
            qs = check_rows(q, "q", device, 4)
            if q.shape != dq_out.shape:
                raise ValueError(f"q must have shape {tuple(dq_out.shape)}, got {tuple(q.shape)}")
        if k is not None:
            if dk_out is None:
                raise ValueError("k without dk_out")
            ks = check_rows(k, "k", device, 4, None if q is None else q.dtype)
            if k.shape != dk_out.shape:
                raise ValueError(f"k must have shape {tuple(dk_out.shape)}, got {tuple(k.shape)}")
        hn = head_norm(norm_eps, q_weight, k_weight, D, device)
        x_dtype = (q if q is not None else k if k is not None else dq_out).dtype
        if dq is None:
            dq = torch.empty_like(dq_out, dtype=x_dtype) if q is None else torch.empty_like(q, dtype=x_dtype)
            os = dq.stride()
        else:
            os = self._check_out(dq, "dq", dq_out, None)
        oks, gk_ptr, dk_ptr = NO_STRIDES, 0, 0
        if dk_out is None:
            dk = None
        else:
            if dk is None:
                dk = torch.empty_like(dk_out if k is None else k, dtype=dq.dtype)
                oks = dk.stride()
            else:
                oks = self._check_out(dk, "dk", dk_out, dq.dtype)
            gk_ptr, dk_ptr = dk_out.data_ptr(), dk.data_ptr()
        dqw = dkw = None
        if q_weight is not None:
            dqw = torch.empty_like(q_weight, dtype=torch.float32)
        if k_weight is not None and Hkv > 0:
            dkw = torch.empty_like(k_weight, dtype=torch.float32)
        fields = (
            B, n, Hq, Hkv, D, _dtype_code(x_dtype), _dtype_code(dq_out.dtype), _dtype_code(dq.dtype),
            0 if q is None else q.data_ptr(), 0 if k is None else k.data_ptr(), qs[0], qs[1], qs[2],
            ks[0], ks[1], ks[2], check_index(positions, "positions", device, (B, n)), start, dq_out.data_ptr(), gk_ptr,
            gs[0], gs[1], gs[2], gks[0], gks[1], gks[2], dq.data_ptr(), dk_ptr, os[0], os[1], os[2], oks[0], oks[1],
            oks[2], 0 if dqw is None else dqw.data_ptr(), 0 if dkw is None else dkw.data_ptr(), *self.fields, *hn)
        ws, need = 0, 0
        if dqw is not None or dkw is not None:
            need = self._lib.swa_rotary_workspace_bytes(_pack_backward(*fields, 0, 0))
            space = torch.empty(need, dtype=torch.uint8, device=device)
            ws = space.data_ptr()
        st = self._lib.swa_rotary_backward(_pack_backward(*fields, ws, need), current_stream(dq_out))
        if st != 0:
            raise SwaError(st, "swa_rotary_backward")
        return (dq, dk) if norm_eps is None else (dq, dk, dqw, dkw)

    @staticmethod
    def _check_out(t, name, like, dtype=0):
        strides = check_rows(t, name, like.device, 4, like.dtype if dtype == 0 else dtype)
        if t.shape != like.shape:
            raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
        return strides
