"""The dense operators of a handle: norm, linear layers and distillation.

Argument marshalling only, like the rest of the binding: torch tensors become
pointers and sizes, outputs and scratch are torch tensors allocated on the
call's stream.  Matrices are 2-D with contiguous rows (any stride between
rows); vectors are 1-D and contiguous.  The formulas stand in
``include/sparsecos.h``.
"""
from __future__ import annotations

import contextlib
from typing import Optional, Tuple

import torch

from . import _abi

_TYPES = {torch.float32: _abi.SS_VALUES_F32, torch.bfloat16: _abi.SS_VALUES_BF16,
          torch.float16: _abi.SS_VALUES_F16, torch.float8_e4m3fn: _abi.SS_VALUES_F8}
ACTIVATIONS = {"none": _abi.SS_ACT_NONE, "relu": _abi.SS_ACT_RELU, "gelu": _abi.SS_ACT_GELU,
               "gelu_tanh": _abi.SS_ACT_GELU_TANH, "silu": _abi.SS_ACT_SILU,
               "log1p_relu": _abi.SS_ACT_LOG1P_RELU}
_NOTHING = contextlib.nullcontext()


def _on(stream: Optional[torch.cuda.Stream]):
    """Allocations inside belong to the stream that the call runs on."""
    return _NOTHING if stream is None else torch.cuda.stream(stream)


class DenseOperators:
    """Mixed into SparseCosine: calls that share its handle, device and errors."""

    def _matrix(self, t: Optional[torch.Tensor], name: str):
        if t is None:
            return None
        if not t.is_cuda or t.device.index != self.device:
            raise ValueError(f"{name} is on {t.device}, the handle's device is cuda:{self.device}")
        code = _TYPES.get(t.dtype)
        if code is None:
            raise TypeError(f"{name} has type {t.dtype}")
        shape, stride = t.shape, t.stride()
        if len(shape) == 2:
            if shape[1] > 1 and stride[1] != 1:
                raise ValueError(f"{name}: the values of a row must be contiguous")
            return _abi.ss_dense(t.data_ptr(), shape[0], shape[1],
                                 stride[0] if shape[0] > 1 else shape[1], code)
        if len(shape) == 1:
            if shape[0] > 1 and stride[0] != 1:
                raise ValueError(f"{name} must be contiguous")
            return _abi.ss_dense(t.data_ptr(), 1, shape[0], shape[0], code)
        raise ValueError(f"{name} must be a matrix or a vector, got {len(shape)} dimensions")

    def _vector(self, t: Optional[torch.Tensor], name: str, shape: Tuple[int, ...], dtype=torch.float32):
        """The address of a contiguous array of the given shape and type."""
        if t is None:
            return None
        if not t.is_cuda or t.device.index != self.device:
            raise ValueError(f"{name} is on {t.device}, the handle's device is cuda:{self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} has type {t.dtype}, expected {dtype}")
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous array of shape {shape}, got {tuple(t.shape)}")
        return t.data_ptr()

    @staticmethod
    def _stream(stream: Optional[torch.cuda.Stream], like: torch.Tensor) -> int:
        return (stream if stream is not None else torch.cuda.current_stream(like.device)).cuda_stream

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
        mx, mr, mw = self._matrix(x, "x"), self._matrix(residual, "residual"), self._matrix(weight, "weight")
        with _on(stream):
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            total = x if residual is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
            rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        mt = None if residual is None else self._matrix(total, "total")
        self._check(self._lib.ss_rms_norm(self._h, mx, mr, mw, eps, mt, self._matrix(y, "y"), None, rstd.data_ptr(),
                                          self._stream(stream, x)), "ss_rms_norm")
        return y, total, rstd

    def rms_norm_quantized(self, x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                           eps: float = 1e-6, stream=None):
        """(y, scale, total): as ``rms_norm`` with y in e4m3 and one float32
        scale a row (the norm is y * scale), as ``linear`` takes them."""
        mx, mr, mw = self._matrix(x, "x"), self._matrix(residual, "residual"), self._matrix(weight, "weight")
        with _on(stream):
            y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
            total = x if residual is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
            scale = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        mt = None if residual is None else self._matrix(total, "total")
        self._check(self._lib.ss_rms_norm(self._h, mx, mr, mw, eps, mt, self._matrix(y, "y"), scale.data_ptr(), None,
                                          self._stream(stream, x)), "ss_rms_norm")
        return y, scale, total

    def rms_norm_backward(self, grad_y: torch.Tensor, total: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          grad_total: Optional[torch.Tensor] = None, stream=None):
        """(grad_x, grad_weight); grad_x is the residual's gradient too.
        grad_total: the gradient that reaches total past the norm."""
        mg, mt, mw = self._matrix(grad_y, "grad_y"), self._matrix(total, "total"), self._matrix(weight, "weight")
        mp = self._matrix(grad_total, "grad_total")
        pr = self._vector(rstd, "rstd", (total.shape[0],))
        with _on(stream):
            gx = torch.empty(total.shape, dtype=total.dtype, device=total.device)
            gw = torch.empty(weight.shape, dtype=weight.dtype, device=total.device)
            keep, at, n = self._scratch(self._lib.ss_rms_norm_backward_scratch(self._h, mt.n_rows, mt.n_cols), total)
        self._check(self._lib.ss_rms_norm_backward(self._h, mg, mt, mw, pr, mp, self._matrix(gx, "grad_x"),
                                                   self._matrix(gw, "grad_weight"), at, n,
                                                   self._stream(stream, total)), "ss_rms_norm_backward")
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
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
        mx, mw, mr = self._matrix(x, "x"), self._matrix(w, "w"), self._matrix(residual, "residual")
        m, n = mx.n_rows, mw.n_rows
        if out_dtype is None:
            out_dtype = torch.bfloat16 if x.dtype == torch.float8_e4m3fn else x.dtype
        sx, sw = self._vector(x_scale, "x_scale", (m,)), self._vector(w_scale, "w_scale", (n,))
        pb = self._vector(bias, "bias", (n,))
        with _on(stream):
            y = torch.empty((m, n), dtype=out_dtype, device=x.device)
            pre = torch.empty((m, n), dtype=out_dtype, device=x.device) if save_pre else None
            keep, at, size = self._scratch(self._lib.ss_linear_scratch(self._h, mx, mw), x)
        self._check(self._lib.ss_linear(self._h, mx, sx, mw, sw, pb, ACTIVATIONS[activation], mr,
                                        self._matrix(pre, "pre"), self._matrix(y, "y"), at, size,
                                        self._stream(stream, x)), "ss_linear")
        return (y, pre) if save_pre else y

    def linear_backward(self, grad_y: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                        pre: Optional[torch.Tensor] = None, activation: str = "none",
                        grad_dtype: Optional[torch.dtype] = None, stream=None):
        """(grad_x, grad_w, grad_bias) of ``linear`` for 16-bit x and w; pre as
        it kept it (not needed for activation "none").  grad_dtype: of grad_x
        and grad_w, x's type or float32; grad_bias is float32.  The residual's
        gradient is grad_y."""
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
        mg, mx, mw = self._matrix(grad_y, "grad_y"), self._matrix(x, "x"), self._matrix(w, "w")
        mp, act = self._matrix(pre, "pre"), ACTIVATIONS[activation]
        dt = x.dtype if grad_dtype is None else grad_dtype
        with _on(stream):
            gx = torch.empty(x.shape, dtype=dt, device=x.device)
            gw = torch.empty(w.shape, dtype=dt, device=x.device)
            gb = torch.empty(mw.n_rows, dtype=torch.float32, device=x.device)
            keep, at, n = self._scratch(self._lib.ss_linear_backward_scratch(self._h, mg, mx, mw, act), x)
        self._check(self._lib.ss_linear_backward(self._h, mg, mx, mw, mp, act, self._matrix(gx, "grad_x"),
                                                 self._matrix(gw, "grad_w"), gb.data_ptr(), at, n,
                                                 self._stream(stream, x)), "ss_linear_backward")
        return gx, gw, gb

    # -- distillation
    def _lists(self, logits, scores, items, weight):
        ml = self._matrix(logits, "logits")
        if scores.dim() != 2:
            raise ValueError("scores must be (rows, k)")
        rows, k = ml.n_rows, int(scores.shape[1])
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
        self._check(self._lib.ss_distill(self._h, ml, ps, pi, k, temperature, u, pw, loss.data_ptr(),
                                         stats.data_ptr(), self._stream(stream, logits)), "ss_distill")
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
        self._check(self._lib.ss_distill_backward(self._h, pg, ml, ps, pi, k, temperature, u, pw, pt,
                                                  self._matrix(grad, "grad_logits"), self._stream(stream, logits)),
                    "ss_distill_backward")
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
        self._check(self._lib.ss_distill_step(self._h, pg, ml, ps, pi, k, temperature, u, pw, loss.data_ptr(),
                                              ml if in_place else self._matrix(grad, "grad_logits"),
                                              self._stream(stream, logits)), "ss_distill_step")
        return loss, grad
