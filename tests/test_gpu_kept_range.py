"""GPU tests of kept values at and past the ends of the type that the gradients
are computed in: one rule for them, expand's."""
import pytest

torch = pytest.importorskip("torch")

import dense_reference as dense  # noqa: E402
from dense_reference import F64, ROUND, STEP  # noqa: E402

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]
HALVES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_embedding_exact_gb300 as sec
    from sparse_embedding_exact_gb300 import build

    build.build()
    with sec.SparseCosine(1000, chunk_rows=256) as handle:
        yield handle
        handle.check_device()


def _randn(*shape, std=1.0, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def _values(rows, cols, low, high, seed=0):
    """float32 values of sizes from 2^low to 2^high, group by group, each type's
    largest and what lies below its smallest normal among them where they are
    of such sizes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    groups = (cols + 31) // 32
    e = torch.randint(low, high + 1, (rows, groups), device="cuda", generator=g).to(F64).repeat_interleave(32, 1)[:, :cols]
    x = (torch.randn(rows, cols, device="cuda", generator=g).to(F64).clamp(-3, 3) / 4 * torch.exp2(e)).float()
    for k, t in enumerate(TYPES):
        for at, v in ((k, torch.finfo(t).max), (8 * k + 40, torch.finfo(t).smallest_normal / 8)):
            if 2.0 ** (low - 4) <= v <= 2.0 ** (high + 1):
                x[:, at::50] = v * (1 - 2 * (k % 2))
    return x


def _out(want, dtype, extra):
    return ROUND[dtype] * (want.abs() + extra) + extra + STEP[dtype]


def _near(got, want, room, dtype):
    """Within the bound; past the type's largest, where the bound allows it, infinite."""
    got, top = got.to(F64), torch.finfo(dtype).max
    fine = torch.isfinite(got)
    assert not torch.isnan(got).any()
    assert ((got - want).abs() <= room)[fine].all() and (want.abs() + room >= top)[~fine].all()


# Sizes of values and the row's factor that brings them near 1 (or, for the
# smallest, as near as its square allows): at the ends of float32 and bfloat16, at
# those of float16.
SIZES = [(100, 127, 2.0 ** -120), (8, 18, 2.0 ** -14), (-30, -8, 2.0 ** 8), (-140, -110, 2.0 ** 60)]


# The widest row that its kernel keeps in registers, the ones beyond it (by way
# of a widened copy), and rows of units and of single values.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kept", TYPES)
@pytest.mark.parametrize("rows,cols", [(3, 64), (5, 101), (300, 1024), (3, 8191), (3, 8192), (3, 8200)])
def test_a_norms_total(h, dtype, kept, rows, cols):
    for low, high, std in SIZES:
        top = torch.finfo(kept).max
        q, s = h.compress(_values(rows, cols, low, high).clamp(-top, top).to(kept))
        v = h.expand(q, s, dtype).to(F64)
        rstd, w = torch.full((rows,), std, device="cuda"), _randn(cols, seed=1)
        gy, gt = _randn(rows, cols, dtype=dtype, seed=2), _randn(rows, cols, dtype=dtype, seed=3)
        gx, gw = h.rms_norm_backward(gy, q, w, rstd, gt, total_scale=s)
        wx, ww = dense.rms_norm_grad(gy, v, w, rstd, gt)
        xh, g = v.abs() * std, gy.to(F64).abs() * w.to(F64).abs()
        size = std * (g + xh * (g * xh).mean(1, keepdim=True)) + gt.to(F64).abs()
        # products of small values and factors fall below float32's smallest
        _near(gx, wx, _out(wx, dtype, 64 * E * size + 2.0 ** -120), dtype)
        wsize = (gy.to(F64).abs() * xh).sum(0)
        _near(gw, ww, _out(ww, torch.float32, (64 + rows / 8) * E * wsize + 2.0 ** -120), torch.float32)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("kept", TYPES)
@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu", "log1p_relu"])
@pytest.mark.parametrize("n", [256, 333])
def test_a_layers_pre_activation(h, dtype, kept, name, n):
    """The gradients from the codes are those from the values that expand gives."""
    m, k = 70, 64
    top = torch.finfo(kept).max
    pre = torch.cat([_values(14, n, low, high) for low, high, _ in SIZES] + [_randn(14, n, std=3.0, seed=4)]).clamp(-top, top).to(kept)
    x, w, gy = _randn(m, k, dtype=dtype), _randn(n, k, dtype=dtype, seed=1), _randn(m, n, dtype=dtype, seed=2)
    q, s = h.compress(pre)
    got = h.linear_backward(gy, x, w, q, name, pre_scale=s)
    want = h.linear_backward(gy, x, w, h.expand(q, s, dtype), name)
    for a, b in zip(got, want):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("name", ["gelu", "log1p_relu", "silu"])
def test_pre_activations_past_float16(h, name):
    """A layer's z beyond float16's largest is kept as that."""
    m, k, n, dtype = 40, 64, 96, torch.float16
    x, w = torch.full((m, k), 64.0, device="cuda", dtype=dtype), torch.ones(n, k, device="cuda", dtype=dtype)
    b = torch.linspace(-9e4, 9e4, n, device="cuda")
    _, q, s = h.linear(x, w, bias=b, activation=name, compress_pre=True)
    gy = _randn(m, n, dtype=dtype, seed=2)
    got = h.linear_backward(gy, x, w, q, name, pre_scale=s)
    v = h.expand(q, s, dtype)
    assert float(v.abs().max()) == 65504
    for a, c in zip(got, h.linear_backward(gy, x, w, v, name)):
        assert torch.equal(a, c)
