"""GPU tests of the dense operators where values or sizes reach a limit: zero
rows without eps, scales far from 1, the activations' tails.

Tolerances are bounds, not fits, of the kernels' float32 steps (unit roundoff
E = 2^-24 each).
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
F64 = torch.float64
F8 = torch.float8_e4m3fn
TYPES = [torch.float32, torch.bfloat16, torch.float16]


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


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [7, 256, 1001, 20000, 33001])
def test_zero_row_to_8_bits_without_eps(h, dtype, cols):
    x = _randn(3, cols, dtype=dtype)
    x[1] = 0
    y, scale, _ = h.rms_norm_quantized(x, torch.ones(cols, device="cuda"), eps=0.0)
    assert float(scale[1]) == 0 and not y[1].float().any()
    assert torch.isfinite(scale).all() and (scale[[0, 2]] > 0).all()
    assert (y[[0, 2]].float().abs().amax(1) == 448).all()


# ---------------------------------------------------------------- linear
# One row; few rows (features along the tile's rows); one tile; many tiles, an
# odd row length and rows of features off 16 bytes.
SCALE_SHAPES = [(1, 64, 96), (16, 256, 300), (40, 4096, 256), (300, 256, 520), (300, 200, 333), (2600, 64, 4000)]


@pytest.mark.parametrize("m,k,n", SCALE_SHAPES)
@pytest.mark.parametrize("sx,sw,x", [(1e-25, 1e-20, 448.0), (1e25, 1e16, 2.0 ** -9), (1e-19, 1e-30, 448.0)])
def test_row_scales_apply_one_after_the_other(h, m, k, n, sx, sw, x):
    # Every sum is k x^2, exact in float32 (448^2 = 49 * 2^12, k below 2^13);
    # the scales' product alone would be 0 or infinite.
    one = torch.full((m, k), x, device="cuda")
    one[m // 2] = 0  # a row of zeros: 0 whatever the scales are
    a, b = one.to(F8), torch.full((n, k), x, device="cuda").to(F8)
    vx, vw = torch.full((m,), sx, device="cuda"), torch.full((n,), sw, device="cuda")
    y = h.linear(a, b, x_scale=vx, w_scale=vw, out_dtype=torch.float32)
    want = (a.to(F64) @ b.to(F64).t() * vx.to(F64)[:, None] * vw.to(F64))
    fits = want <= torch.finfo(torch.float32).max  # past it the float32 output is infinite
    # two roundings, and results below 2^-126 keep a step of 2^-149
    assert ((y.to(F64) - want).abs() <= 2 * E * want.abs() + 2.0 ** -149)[fits].all()
    assert torch.isinf(y[~fits]).all() and not y[m // 2].any()


@pytest.mark.parametrize("k", [64, 100])
def test_row_scales_of_one_row(h, k):
    x, w = torch.full((1, k), 448.0, device="cuda").to(F8), torch.full((77, k), 448.0, device="cuda").to(F8)
    sx, sw = torch.full((1,), 1e-30, device="cuda"), torch.full((77,), 1e-19, device="cuda")
    y = h.linear(x, w, x_scale=sx, w_scale=sw, out_dtype=torch.float32)
    want = x.to(F64) @ w.to(F64).t() * sx.to(F64)[:, None] * sw.to(F64)
    assert ((y.to(F64) - want).abs() <= 2 * E * want.abs() + 2.0 ** -149).all() and (y > 0).all()


# ---------------------------------------------------------------- activations
# In multiples of E, relative to the result; z reaches the activation exactly
# (as the bias of rows of zeros).  An exponential of an argument of size a has
# the argument's two or three roundings, 2.5 a E at most, and the instruction's
# 4 E; the rest is a dozen roundings, their factors below 2, and the
# polynomial's 3 E.
TAILS = {
    "gelu": (lambda z: 0.5 * torch.erfc(-z / 2 ** 0.5), lambda z: 1.25 * z * z + 24),
    "gelu_tanh": (lambda z: 1 / (1 + torch.exp(-2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))),
                  lambda z: 6 * (2 / torch.pi) ** 0.5 * (z.abs() + 0.044715 * z.abs() ** 3) + 24),
    "silu": (lambda z: 1 / (1 + torch.exp(-z)), lambda z: 3 * z.abs() + 24),
}


def _tail(name, m):
    """act(z) of m rows for z from -8 to -2 and a few around 0, in 64 bits too."""
    z = torch.cat([torch.linspace(-8, -2, 1200), torch.linspace(-2, 3, 336)]).cuda()
    x, w = torch.zeros(m, 64, dtype=torch.bfloat16, device="cuda"), _randn(z.numel(), 64, dtype=torch.bfloat16)
    share, units = TAILS[name]
    return x, w, z, share(z.to(F64)), units(z.to(F64)) * E


def _tail_of(h, name, m, dtype):
    x, w, z, share, room = _tail(name, m)
    want = z.to(F64) * share
    y = h.linear(x.to(dtype) if dtype != torch.float32 else x, w.to(dtype) if dtype != torch.float32 else w, bias=z,
                 activation=name, out_dtype=dtype)
    return y.to(F64), want, room


@pytest.mark.parametrize("m", [1, 40, 600])
def test_gelu_of_negative_values(h, m):
    y, want, room = _tail_of(h, "gelu", m, torch.float32)
    assert ((y - want).abs() <= (room + E) * want.abs()).all()
    y, want, room = _tail_of(h, "gelu", m, torch.bfloat16)
    assert ((y - want).abs() <= (room + 2.0 ** -8) * want.abs()).all()
    y, want, room = _tail_of(h, "gelu", m, torch.float16)
    assert ((y - want).abs() <= (room + 2.0 ** -11) * want.abs() + 2.0 ** -25).all()


@pytest.mark.parametrize("m", [1, 40, 600])
@pytest.mark.parametrize("name", ["gelu_tanh", "silu"])
def test_gelu_tanh_and_silu_of_negative_values(h, name, m):
    y, want, room = _tail_of(h, name, m, torch.float32)
    assert ((y - want).abs() <= (room + E) * want.abs()).all()
    y, want, room = _tail_of(h, name, m, torch.bfloat16)
    assert ((y - want).abs() <= (room + 2.0 ** -8) * want.abs()).all()
    y, want, room = _tail_of(h, name, m, torch.float16)
    assert ((y - want).abs() <= (room + 2.0 ** -11) * want.abs() + 2.0 ** -25).all()


@pytest.mark.parametrize("name", ["gelu_tanh", "silu", "gelu"])
def test_slopes_of_large_values(h, name):
    # grad_bias of one row is grad_y act'(pre): 0 or 1 where the activation is
    # flat or the identity, and finite everywhere
    z = torch.tensor([-1e38, -1e20, -3e4, -300.0, -90.0, -88.0, 88.0, 300.0, 3e4, 1e38], device="cuda").to(torch.bfloat16)
    n = z.numel()
    gy = torch.ones(1, n, dtype=torch.bfloat16, device="cuda")
    x, w = torch.ones(1, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(n, 16, dtype=torch.bfloat16, device="cuda")
    _, _, gb = h.linear_backward(gy, x, w, z[None], name)
    assert ((gb - (z > 0).float()).abs() <= 1e-30).all()
    y = h.linear(torch.zeros(1, 16, dtype=torch.bfloat16, device="cuda"), w, bias=z.float(), activation=name, out_dtype=torch.float32)
    assert ((y[0] - torch.relu(z.float())).abs() <= 1e-30).all()
