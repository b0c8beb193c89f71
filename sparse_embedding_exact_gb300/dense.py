"""The dense operators of a handle: norm, linear layers and distillation.

Argument marshalling only, like the rest of the binding: torch tensors become
pointers and sizes, outputs and scratch are torch tensors allocated on the
call's stream.  Matrices are 2-D with contiguous rows (any stride between
rows); vectors are 1-D and contiguous.  The formulas stand in
``include/sparsecos.h``.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct
from typing import Optional, Tuple

import torch

from . import _abi

_TYPES = {torch.float32: _abi.SS_VALUES_F32, torch.bfloat16: _abi.SS_VALUES_BF16,
          torch.float16: _abi.SS_VALUES_F16, torch.float8_e4m3fn: _abi.SS_VALUES_F8}
ACTIVATIONS = {"none": _abi.SS_ACT_NONE, "relu": _abi.SS_ACT_RELU, "gelu": _abi.SS_ACT_GELU,
               "gelu_tanh": _abi.SS_ACT_GELU_TANH, "silu": _abi.SS_ACT_SILU,
               "log1p_relu": _abi.SS_ACT_LOG1P_RELU}
_F8 = torch.float8_e4m3fn
_NOTHING = contextlib.nullcontext()
# A call's matrices are packed as ss_dense records side by side, in one call of
# struct: short calls cost their host time, and ctypes structures are slow.
_SIZE = ctypes.sizeof(_abi.ss_dense)
_PACK = [struct.Struct("@" + "qqqqi4x" * n).pack_into for n in range(8)]
assert _SIZE == struct.calcsize("@qqqqi4x")


def _on(stream: Optional[torch.cuda.Stream]):
    """Allocations inside belong to the stream that the call runs on."""
    return _NOTHING if stream is None else torch.cuda.stream(stream)


class DenseOperators:
    """Mixed into SparseCosine: calls that share its handle, device and errors."""

    def _records(self, *fields):
        """The addresses of ss_dense records of the given fields (five a
        record), valid until the handle's next call."""
        if not hasattr(self, "_record_buf"):
            self._record_buf = ctypes.create_string_buffer(_SIZE * 7)
            at = ctypes.addressof(self._record_buf)
            self._record_at = [at + k * _SIZE for k in range(7)]
        _PACK[len(fields) // 5](self._record_buf, 0, *fields)
        return self._record_at

    def _matrix(self, t: torch.Tensor, name: str):
        """(address, rows, columns, values a row, type) of a matrix, or of a
        vector as one row."""
        if t.get_device() != self.device:
            raise ValueError(f"{name} is on {t.device}, the handle's device is cuda:{self.device}")
        code = _TYPES.get(t.dtype)
        if code is None:
            raise TypeError(f"{name} has type {t.dtype}")
        shape = t.shape
        if t.is_contiguous():
            if len(shape) == 2:
                rows, cols = shape
                return t.data_ptr(), rows, cols, cols, code
            if len(shape) == 1:
                cols = shape[0]
                return t.data_ptr(), 1, cols, cols, code
        elif len(shape) == 2:
            rows, cols = shape
            if cols <= 1 or t.stride(1) == 1:
                return t.data_ptr(), rows, cols, t.stride(0) if rows > 1 else cols, code
            raise ValueError(f"{name}: the values of a row must be contiguous")
        elif len(shape) == 1:
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} must be a matrix or a vector, got {len(shape)} dimensions")

    def _vector(self, t: Optional[torch.Tensor], name: str, shape: Tuple[int, ...], dtype=torch.float32):
        """The address of a contiguous array of the given shape and type."""
        if t is None:
            return None
        if t.get_device() != self.device:
            raise ValueError(f"{name} is on {t.device}, the handle's device is cuda:{self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} has type {t.dtype}, expected {dtype}")
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous array of shape {shape}, got {tuple(t.shape)}")
        return t.data_ptr()

    def _where(self, stream: Optional[torch.cuda.Stream]) -> int:
        """The stream's handle: the given one's or the current one's."""
        return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(self.device)

    @staticmethod
    def _scratch(n: int, like: torch.Tensor):
        """(tensor, address, bytes) of scratch; torch aligns to 512 bytes."""
        if n == 0:
            return None, None, 0
        t = torch.empty(n, dtype=torch.uint8, device=like.device)
        return t, t.data_ptr(), n

    # -- norm
    def rms_norm(self, x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, stream=None):
        """(y, total, rstd): the norm of x + residual, that sum (x itself
        without a residual) and the float32 factor of each row; total and rstd
        are what ``rms_norm_backward`` takes."""
        return self._norm(x, weight, residual, eps, stream, False)

    def rms_norm_quantized(self, x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                           eps: float = 1e-6, stream=None):
        """(y, scale, total): as ``rms_norm`` with y in e4m3 and one float32
        scale a row (the norm is y * scale), as ``linear`` takes them."""
        y, total, scale = self._norm(x, weight, residual, eps, stream, True)
        return y, scale, total

    def _norm(self, x, weight, residual, eps, stream, f8):
        mx = self._matrix(x, "x")
        shape, dev, dt = x.shape, x.device, x.dtype
        rows, cols = mx[1], mx[2]
        with _on(stream):
            y = torch.empty(shape, dtype=_F8 if f8 else dt, device=dev)
            factor = torch.empty(rows, dtype=torch.float32, device=dev)
            total = x if residual is None else torch.empty(shape, dtype=dt, device=dev)
        my = (y.data_ptr(), rows, cols, cols, _abi.SS_VALUES_F8 if f8 else mx[4])
        if residual is None:
            at = self._records(*mx, *self._matrix(weight, "weight"), *my)
            mr = mt = None
        else:
            at = self._records(*mx, *self._matrix(weight, "weight"), *my, *self._matrix(residual, "residual"),
                               total.data_ptr(), rows, cols, cols, mx[4])
            mr, mt = at[3], at[4]
        f = factor.data_ptr()
        st = self._lib.ss_rms_norm(self._h, at[0], mr, at[1], eps, mt, at[2], f if f8 else None, None if f8 else f,
                                   self._where(stream))
        if st:
            self._check(st, "ss_rms_norm")
        return y, total, factor

    def rms_norm_backward(self, grad_y: torch.Tensor, total: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          grad_total: Optional[torch.Tensor] = None, stream=None):
        """(grad_x, grad_weight); grad_x is the residual's gradient too.
        grad_total: the gradient that reaches total past the norm."""
        mt, mw = self._matrix(total, "total"), self._matrix(weight, "weight")
        rows, cols = mt[1], mt[2]
        pr = self._vector(rstd, "rstd", (rows,))
        with _on(stream):
            gx = torch.empty(total.shape, dtype=total.dtype, device=total.device)
            gw = torch.empty(weight.shape, dtype=weight.dtype, device=total.device)
            keep, room, n = self._scratch(self._lib.ss_rms_norm_backward_scratch(self._h, rows, cols), total)
        fields = (*self._matrix(grad_y, "grad_y"), *mt, *mw, gx.data_ptr(), rows, cols, cols, mt[4],
                  gw.data_ptr(), *mw[1:3], mw[2], mw[4])
        if grad_total is None:
            at, mp = self._records(*fields), None
        else:
            at = self._records(*fields, *self._matrix(grad_total, "grad_total"))
            mp = at[5]
        st = self._lib.ss_rms_norm_backward(self._h, at[0], at[1], at[2], pr, mp, at[3], at[4], room, n,
                                            self._where(stream))
        if st:
            self._check(st, "ss_rms_norm_backward")
        return gx, gw

    # -- linear layers
    def linear(self, x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, activation: str = "none",
               residual: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None,
               w_scale: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
               save_pre: bool = False, stream=None):
        """act(x w^T + bias) + residual, x (M, K) and w (N, K) in bfloat16,
        float16, or e4m3 with float32 scales of their rows; bias float32.
        out_dtype: x's type (bfloat16 for e4m3) or float32; residual has it
        too.  With save_pre the pair (y, pre), pre the activation's input as
        ``linear_backward`` takes it."""
        act = ACTIVATIONS.get(activation)
        if act is None:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
        mx, mw = self._matrix(x, "x"), self._matrix(w, "w")
        m, n = mx[1], mw[1]
        if out_dtype is None:
            out_dtype = torch.bfloat16 if mx[4] == _abi.SS_VALUES_F8 else x.dtype
        code = _TYPES.get(out_dtype)
        if code is None:
            raise TypeError(f"out_dtype {out_dtype}")
        sx, sw = self._vector(x_scale, "x_scale", (m,)), self._vector(w_scale, "w_scale", (n,))
        pb = self._vector(bias, "bias", (n,))
        dev = x.device
        with _on(stream):
            y = torch.empty((m, n), dtype=out_dtype, device=dev)
            pre = torch.empty((m, n), dtype=out_dtype, device=dev) if save_pre else None
        fields, mp, mr, k = (*mx, *mw, y.data_ptr(), m, n, n, code), None, None, 3
        if save_pre:
            fields, k = fields + (pre.data_ptr(), m, n, n, code), 4
        if residual is not None:
            fields += self._matrix(residual, "residual")
        at = self._records(*fields)
        if save_pre:
            mp = at[3]
        if residual is not None:
            mr = at[k]
        size = self._lib.ss_linear_scratch(self._h, at[0], at[1])
        room = None
        if size:
            with _on(stream):
                keep, room, size = self._scratch(size, x)
        st = self._lib.ss_linear(self._h, at[0], sx, at[1], sw, pb, act, mr, mp, at[2], room, size,
                                 self._where(stream))
        if st:
            self._check(st, "ss_linear")
        return (y, pre) if save_pre else y

    def linear_backward(self, grad_y: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                        pre: Optional[torch.Tensor] = None, activation: str = "none",
                        grad_dtype: Optional[torch.dtype] = None, stream=None):
        """(grad_x, grad_w, grad_bias) of ``linear`` for 16-bit x and w; pre as
        it kept it (not needed for activation "none").  grad_dtype: of grad_x
        and grad_w, x's type or float32; grad_bias is float32.  The residual's
        gradient is grad_y."""
        act = ACTIVATIONS.get(activation)
        if act is None:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
        mx, mw = self._matrix(x, "x"), self._matrix(w, "w")
        dt = x.dtype if grad_dtype is None else grad_dtype
        code = _TYPES.get(dt)
        if code is None:
            raise TypeError(f"grad_dtype {dt}")
        dev = x.device
        with _on(stream):
            gx = torch.empty(x.shape, dtype=dt, device=dev)
            gw = torch.empty(w.shape, dtype=dt, device=dev)
            gb = torch.empty(mw[1], dtype=torch.float32, device=dev)
        fields = (*self._matrix(grad_y, "grad_y"), *mx, *mw, gx.data_ptr(), mx[1], mx[2], mx[2], code,
                  gw.data_ptr(), mw[1], mw[2], mw[2], code)
        if pre is None:
            at, mp = self._records(*fields), None
        else:
            at = self._records(*fields, *self._matrix(pre, "pre"))
            mp = at[5]
        size = self._lib.ss_linear_backward_scratch(self._h, at[0], at[1], at[2], act)
        with _on(stream):
            keep, room, size = self._scratch(size, x)
        st = self._lib.ss_linear_backward(self._h, at[0], at[1], at[2], mp, act, at[3], at[4], gb.data_ptr(), room, size,
                                          self._where(stream))
        if st:
            self._check(st, "ss_linear_backward")
        return gx, gw, gb

    # -- distillation
    def _lists(self, logits, scores, items, weight):
        ml = self._matrix(logits, "logits")
        if scores.dim() != 2:
            raise ValueError("scores must be (rows, k)")
        rows, k = ml[1], scores.shape[1]
        return (ml, rows, k, self._vector(scores, "scores", (rows, k)),
                self._vector(items, "items", (rows, k), torch.int64), self._vector(weight, "weight", (rows,)))

    def distill(self, logits: torch.Tensor, scores: torch.Tensor, items: torch.Tensor,
                weight: Optional[torch.Tensor] = None, temperature: float = 1.0,
                teacher_temperature: Optional[float] = None, stream=None):
        """(loss, stats): per row weight * T^2 * KL(teacher || student), the
        teacher's softmax over its listed items (``topk_all``'s values and
        items), the student's over all of its logits; stats are what
        ``distill_backward`` takes.  teacher_temperature: T when not given."""
        ml, rows, k, ps, pi, pw = self._lists(logits, scores, items, weight)
        u = temperature if teacher_temperature is None else teacher_temperature
        with _on(stream):
            loss = torch.empty(rows, dtype=torch.float32, device=logits.device)
            stats = torch.empty((rows, 2), dtype=torch.float32, device=logits.device)
        st = self._lib.ss_distill(self._h, self._records(*ml)[0], ps, pi, k, temperature, u, pw, loss.data_ptr(),
                                  stats.data_ptr(), self._where(stream))
        if st:
            self._check(st, "ss_distill")
        return loss, stats

    def distill_backward(self, grad_loss: Optional[torch.Tensor], logits: torch.Tensor, scores: torch.Tensor,
                         items: torch.Tensor, stats: torch.Tensor, weight: Optional[torch.Tensor] = None,
                         temperature: float = 1.0, teacher_temperature: Optional[float] = None,
                         stream=None) -> torch.Tensor:
        """The logits' gradient; grad_loss: float32 of each row's loss (None: 1)."""
        ml, rows, k, ps, pi, pw = self._lists(logits, scores, items, weight)
        u = temperature if teacher_temperature is None else teacher_temperature
        pg, pt = self._vector(grad_loss, "grad_loss", (rows,)), self._vector(stats, "stats", (rows, 2))
        with _on(stream):
            grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        at = self._records(*ml, grad.data_ptr(), rows, ml[2], ml[2], ml[4])
        st = self._lib.ss_distill_backward(self._h, pg, at[0], ps, pi, k, temperature, u, pw, pt, at[1],
                                           self._where(stream))
        if st:
            self._check(st, "ss_distill_backward")
        return grad

    def distill_step(self, logits: torch.Tensor, scores: torch.Tensor, items: torch.Tensor,
                     grad_loss: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                     temperature: float = 1.0, teacher_temperature: Optional[float] = None, in_place: bool = False,
                     stream=None):
        """(loss, grad_logits) in one launch, the logits read once.  in_place:
        the gradient replaces the logits."""
        ml, rows, k, ps, pi, pw = self._lists(logits, scores, items, weight)
        u = temperature if teacher_temperature is None else teacher_temperature
        pg = self._vector(grad_loss, "grad_loss", (rows,))
        with _on(stream):
            loss = torch.empty(rows, dtype=torch.float32, device=logits.device)
            grad = logits if in_place else torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        at = self._records(*ml) if in_place else self._records(*ml, grad.data_ptr(), rows, ml[2], ml[2], ml[4])
        st = self._lib.ss_distill_step(self._h, pg, at[0], ps, pi, k, temperature, u, pw, loss.data_ptr(),
                                       at[0] if in_place else at[1], self._where(stream))
        if st:
            self._check(st, "ss_distill_step")
        return loss, grad
