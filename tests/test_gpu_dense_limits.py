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
