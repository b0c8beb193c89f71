"""The dense operators of a handle: norm, linear layers and distillation.

Matrices are 2-D with contiguous rows (any stride between rows that holds one);
vectors are 1-D and contiguous.  Outputs are new torch tensors on the call's
stream.  The calls stand outside of torch's autograd: inputs may require
gradients, new outputs never do, and the ``_backward`` calls and ``distill_step``
give the gradients (``logits.backward(grad)`` hands one on to torch).  The
formulas stand in ``include/sparsecos.h``; the marshalling is native
(``csrc/binding.cpp``), as a short call is mostly host time.
"""
from __future__ import annotations

import importlib.util
from typing import Optional

import torch

from . import _abi
from . import build as _build

_TYPES = {torch.float32: _abi.SS_VALUES_F32, torch.bfloat16: _abi.SS_VALUES_BF16, torch.float16: _abi.SS_VALUES_F16}
ACTIVATIONS = {"none": _abi.SS_ACT_NONE, "relu": _abi.SS_ACT_RELU, "gelu": _abi.SS_ACT_GELU,
               "gelu_tanh": _abi.SS_ACT_GELU_TANH, "silu": _abi.SS_ACT_SILU,
               "log1p_relu": _abi.SS_ACT_LOG1P_RELU}
_native = None


def _load():
    """The native binding, loaded once; raises if it has not been built, or
    not for this torch."""
    global _native
    if _native is None:
        _abi.load()
        built_for = _build.binding_torch()
        if built_for != str(torch.__version__):
            state = "is not built" if built_for is None else f"was built for torch {built_for}, this is {torch.__version__}"
            raise ImportError(f"the binding of the dense operators ({_build.BINDING}) {state}; "
                              "run python -m sparse_embedding_exact_gb300.build")
        spec = importlib.util.spec_from_file_location("_dense_binding", _build.BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _native = module
    return _native


def _activation(name: str) -> int:
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    return act


def _type(dtype: Optional[torch.dtype]) -> int:
    if dtype is None:
        return -1
    code = _TYPES.get(dtype)
    if code is None:
        raise TypeError(f"outputs are float32, bfloat16 or float16, not {dtype}")
    return code


class DenseOperators:
    """Mixed into SparseCosine: calls that share its handle, device and errors."""

    def _run(self, what: str, stream, *args):
        """One native call, on the current stream or on the given one."""
        call = getattr(_native or _load(), what)
        h = self._h.value if self._h else 0  # a closed handle is refused by the call
        if stream is None:
            out = call(h, self.device, *args)
        else:
            with torch.cuda.stream(stream):
                out = call(h, self.device, *args)
        if type(out) is int:
            self._check(out, "ss_" + ("rms_" if what.startswith("norm") else "") + what)
        return out

    # -- norm
    def rms_norm(self, x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, stream=None):
        """(y, total, rstd): the norm of x + residual, that sum (x itself
        without a residual) and the float32 factor of each row; total and rstd
        are what ``rms_norm_backward`` takes."""
        return self._run("norm", stream, x, weight, residual, eps, False)

    def rms_norm_quantized(self, x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                           eps: float = 1e-6, stream=None):
        """(y, scale, total): as ``rms_norm`` with y in e4m3 and one float32
        scale a row (the norm is y * scale), as ``linear`` takes them."""
        y, total, scale = self._run("norm", stream, x, weight, residual, eps, True)
        return y, scale, total

    def rms_norm_backward(self, grad_y: torch.Tensor, total: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          grad_total: Optional[torch.Tensor] = None, stream=None):
        """(grad_x, grad_weight); grad_x is the residual's gradient too.
        grad_total: the gradient that reaches total past the norm."""
        return self._run("norm_backward", stream, grad_y, total, weight, rstd, grad_total)

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
        return self._run("linear", stream, x, w, bias, _activation(activation), residual, x_scale, w_scale,
                         _type(out_dtype), save_pre)

    def linear_backward(self, grad_y: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                        pre: Optional[torch.Tensor] = None, activation: str = "none",
                        grad_dtype: Optional[torch.dtype] = None, stream=None):
        """(grad_x, grad_w, grad_bias) of ``linear`` for 16-bit x and w; pre as
        it kept it (not needed for activation "none").  grad_dtype: of grad_x
        and grad_w, x's type or float32; grad_bias is float32.  The residual's
        gradient is grad_y."""
        return self._run("linear_backward", stream, grad_y, x, w, pre, _activation(activation), _type(grad_dtype))

    # -- distillation
    def distill(self, logits: torch.Tensor, scores: torch.Tensor, items: torch.Tensor,
                weight: Optional[torch.Tensor] = None, temperature: float = 1.0,
                teacher_temperature: Optional[float] = None, stream=None):
        """(loss, stats): per row weight * T^2 * KL(teacher || student), the
        teacher's softmax over its listed items (``topk_all``'s values and
        items), the student's over all of its logits; stats are what
        ``distill_backward`` takes.  teacher_temperature: T when not given."""
        u = temperature if teacher_temperature is None else teacher_temperature
        return self._run("distill", stream, logits, scores, items, weight, temperature, u)

    def distill_backward(self, grad_loss: Optional[torch.Tensor], logits: torch.Tensor, scores: torch.Tensor,
                         items: torch.Tensor, stats: torch.Tensor, weight: Optional[torch.Tensor] = None,
                         temperature: float = 1.0, teacher_temperature: Optional[float] = None,
                         stream=None) -> torch.Tensor:
        """The logits' gradient; grad_loss: float32 of each row's loss (None: 1)."""
        u = temperature if teacher_temperature is None else teacher_temperature
        return self._run("distill_backward", stream, logits, scores, items, weight, temperature, u, grad_loss, stats)

    def distill_step(self, logits: torch.Tensor, scores: torch.Tensor, items: torch.Tensor,
                     grad_loss: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                     temperature: float = 1.0, teacher_temperature: Optional[float] = None, in_place: bool = False,
                     stream=None):
        """(loss, grad_logits) in one launch, the logits read once.  in_place:
        the gradient replaces the logits, and torch counts them as modified."""
        u = temperature if teacher_temperature is None else teacher_temperature
        return self._run("distill_step", stream, logits, scores, items, weight, temperature, u, grad_loss, in_place)
