"""The 64-bit cross entropy against torch's own and against differences, and the
calls' refusals that need no device."""
import math

import pytest

torch = pytest.importorskip("torch")

import xent_reference as ref  # noqa: E402
from dense_reference import F64  # noqa: E402


def _case(m=7, v=11, k=5, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, k, generator=g), torch.randn(v, k, generator=g), torch.randint(0, v, (m,), generator=g),
            torch.randn(v, generator=g), torch.rand(m, generator=g) + 0.5, torch.randn(m, generator=g))


@pytest.mark.parametrize("T", [0.25, 1.0, 3.0])
def test_against_torch(T):
    x, w, t, b, wt, gl = _case()
    leaves = [a.to(F64).requires_grad_() for a in (x, w, b)]
    loss = wt.to(F64) * torch.nn.functional.cross_entropy((leaves[0] @ leaves[1].t() + leaves[2]) / T, t, reduction="none")
    grads = torch.autograd.grad((loss * gl.to(F64)).sum(), leaves)
    r = ref.cross_entropy(x, w, t, gl, b, wt, T)
    assert (r["loss"] - loss).abs().max() <= 1e-13
    for name, want in zip(("grad_x", "grad_w", "grad_bias"), grads):
        assert (r[name] - want).abs().max() <= 1e-12


def test_gradient_by_differences():
    x, w, t, b, wt, gl = _case(seed=1)
    t[2], wt[4] = -1, 0.0
    b[5] = -math.inf
    t[0] = 5  # a masked target
    r = ref.cross_entropy(x, w, t, gl, b, wt, 0.7)
    assert not r["live"][[0, 2, 4]].any() and r["loss"][[0, 2, 4]].abs().max() == 0
    assert not r["grad_bias"][5] and not r["grad_w"][5].any() and not r["grad_x"][[0, 2, 4]].any()
    f = {0: lambda a: ref.cross_entropy(a, w, t, gl, b, wt, 0.7)["loss"], 1: lambda a: ref.cross_entropy(x, a, t, gl, b, wt, 0.7)["loss"],
         2: lambda a: ref.cross_entropy(x, w, t, gl, a, wt, 0.7)["loss"]}
    for i, (at, name) in enumerate(((x, "grad_x"), (w, "grad_w"), (b, "grad_bias"))):
        d = torch.randn(at.shape, generator=torch.Generator().manual_seed(i), dtype=F64)
        s = 1e-6
        up, down = ((gl.to(F64) * f[i](at.to(F64) + q * s * d)).sum() for q in (1, -1))
        assert abs(float((up - down) / (2 * s) - (r[name] * d).sum())) <= 1e-7


def test_absent_rows_hold_anything():
    x, w, t, b, wt, gl = _case()
    t[1] = -1
    clean = ref.cross_entropy(x, w, t, gl, b, wt)
    x[1] = math.nan
    r = ref.cross_entropy(x, w, t, gl, b, wt)
    for name in ("loss", "grad_x", "grad_w", "grad_bias"):
        assert torch.equal(r[name], clean[name])


def test_a_planted_mistake_is_over_the_bounds():
    x, w, t, b, wt, gl = _case(40, 300, 24)
    x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    r = ref.cross_entropy(x, w, t, gl, b, wt)
    room = ref.bounds(r, x, w, b, wt, gl)
    for wrong in (ref.cross_entropy(x, w, (t + 1) % 300, gl, b, wt), ref.cross_entropy(x, w, t, gl, None, wt),
                  ref.cross_entropy(x, w, t, gl, b, wt, 1.1)):
        for name in ("loss", "grad_x", "grad_w", "grad_bias"):
            assert ((wrong[name] - r[name]).abs() > room[name]).any(), name


def test_calls_without_a_handle_are_refused():
    from sparse_embedding_exact_gb300 import _abi, build

    build.build()
    lib, bad = _abi.load(), _abi.SS_ERR_INVALID_ARG
    assert lib.ss_cross_entropy(None, None, None, None, None, 1.0, None, None, None, None, 0, None) == bad
    assert lib.ss_cross_entropy_backward(None, None, None, None, None, None, 1.0, None, None, None, None, None, None, 0, None) == bad
    assert lib.ss_cross_entropy_step(None, None, None, None, None, None, 1.0, None, None, None, None, None, None, 0, None) == bad
    for call in (lib.ss_cross_entropy_scratch, lib.ss_cross_entropy_backward_scratch, lib.ss_cross_entropy_step_scratch):
        assert call(None, None, None) == 0
