"""The 64-bit forms that the GPU tests compare with: their gradients against
central differences, and against torch's own derivatives."""
import math

import pytest

torch = pytest.importorskip("torch")

import dense_reference as ref  # noqa: E402

F64 = torch.float64
# Central differences of step h err by h^2 times the third derivative (of order
# 10 here) and by 2^-53 / h of rounding: below 1e-8 for h = 1e-5.
H, TOL = 1e-5, 1e-7


def _differences(f, x):
    g = torch.zeros_like(x)
    flat = x.reshape(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + H
        up = float(f())
        flat[i] = keep - H
        down = float(f())
        flat[i] = keep
        g.reshape(-1)[i] = (up - down) / (2 * H)
    return g


def _random(*shape, seed=0):
    return torch.randn(*shape, dtype=F64, generator=torch.Generator().manual_seed(seed))


def test_rms_norm_gradient():
    x, w, gy, gt = _random(3, 7), _random(7, seed=1), _random(3, 7, seed=2), _random(3, 7, seed=3)
    def f():
        y, s, _ = ref.rms_norm(x, w)
        return (gy * y).sum() + (gt * s).sum()
    _, s, rstd = ref.rms_norm(x, w)
    gx, gw = ref.rms_norm_grad(gy, s, w, rstd, gt)
    assert (gx - _differences(f, x)).abs().max() <= TOL
    assert (gw - _differences(f, w)).abs().max() <= TOL


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu", "log1p_relu"])
def test_linear_gradient(name):
    x, w, b, gy = _random(4, 5), _random(3, 5, seed=1), _random(3, seed=2), _random(4, 3, seed=3)
    def f():
        return (gy * ref.linear(x, w, b, name)[0]).sum()
    _, pre, _ = ref.linear(x, w, b, name)
    gx, gw, gb, _ = ref.linear_grad(gy, x, w, pre, name)
    for got, at in ((gx, x), (gw, w), (gb, b)):
        assert (got - _differences(f, at)).abs().max() <= TOL


@pytest.mark.parametrize("T,U", [(1.0, 1.0), (0.5, 2.0), (2.0, 0.25)])
def test_distill_gradient(T, U):
    z, score = _random(3, 11), _random(3, 4, seed=1).float()
    items = torch.tensor([[0, 3, 5, 10], [2, 2, -1, 7], [4, 1, 11, 9]])  # a duplicate, an absent one, one past the end
    weight, gl = torch.tensor([1.0, 0.5, 2.0]), torch.tensor([1.0, -3.0, 0.25])
    def f():
        return (ref.distill(z, score, items, weight, gl, T, U)[0] * gl.to(F64)).sum()
    grad = ref.distill(z, score, items, weight, gl, T, U)[1]
    assert (grad - _differences(f, z)).abs().max() <= TOL


def test_distill_rows_without_anything():
    z = _random(4, 6)
    z[1] = -math.inf
    score, items = torch.zeros(4, 2), torch.tensor([[-1, -1], [0, 1], [0, 1], [2, 3]])
    score[2] = -math.inf
    loss, grad, _, _ = ref.distill(z, score, items, torch.tensor([1.0, 1.0, 1.0, 0.0]))
    assert not loss.any() and not grad.any()


def test_distill_is_zero_for_equal_distributions():
    z = _random(2, 5)
    items = torch.arange(5).repeat(2, 1)
    loss, grad, _, _ = ref.distill(z, z.float(), items)
    assert loss.abs().max() <= 1e-12 and grad.abs().max() <= 1e-6


def test_calls_without_a_handle_are_refused():
    from sparse_embedding_exact_gb300 import _abi, build

    build.build()
    lib, bad = _abi.load(), _abi.SS_ERR_INVALID_ARG
    assert lib.ss_rms_norm(None, None, None, None, 1e-6, None, None, None, None, None) == bad
    assert lib.ss_rms_norm_backward(None, None, None, None, None, None, None, None, None, 0, None) == bad
    assert lib.ss_linear(None, None, None, None, None, None, 0, None, None, None, None, 0, None) == bad
    assert lib.ss_linear_backward(None, None, None, None, None, 0, None, None, None, None, 0, None) == bad
    assert lib.ss_distill(None, None, None, None, 1, 1.0, 1.0, None, None, None, None) == bad
    assert lib.ss_distill_backward(None, None, None, None, None, 1, 1.0, 1.0, None, None, None, None) == bad
    assert lib.ss_distill_step(None, None, None, None, None, 1, 1.0, 1.0, None, None, None, None) == bad
    assert lib.ss_rms_norm_backward_scratch(None, 5, 5) == 0
    assert lib.ss_linear_scratch(None, None, None) == 0
    assert lib.ss_linear_backward_scratch(None, None, None, None, 0) == 0
