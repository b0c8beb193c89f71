"""GPU tests of an activation's slope far out."""
import pytest

torch = pytest.importorskip("torch")

import dense_reference as dense  # noqa: E402
from dense_reference import F64  # noqa: E402

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


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


# The slope reaches grad_bias unrounded where there is one row and grad_y is 1.
# It is s (1 + z (1 - s)), s = 1 / (1 + exp(-z)): the exponential's argument has
# two roundings, 1.5 |z| E at most in the exponential, the instruction 4 E, the
# rest a dozen roundings, and z = -1.278 aside, where the sum in brackets is
# near 0, no cancellation: past -2 the bracket is z's size.  A quotient below
# 2^-126 keeps a step of 2^-149, which the bracket makes |z| 2^-149.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [512, 509])
def test_silu_of_far_negative_values(h, dtype, n):
    z = torch.linspace(-88.5, -2.5, n).cuda().to(dtype)[None]
    gy = torch.ones(1, n, device="cuda", dtype=dtype)
    x, w = torch.ones(1, 8, device="cuda", dtype=dtype), torch.ones(n, 8, device="cuda", dtype=dtype)
    _, _, gb = h.linear_backward(gy, x, w, z, "silu")
    want = dense.act_grad(z.to(F64), "silu")[0]
    room = (3 * z[0].to(F64).abs() + 24) * E * want.abs() + z[0].to(F64).abs() * 2.0 ** -148
    assert ((gb.to(F64) - want).abs() <= room).all()
    assert (gb < 0).all()
