"""The many-row form of the distillation gives what the row-by-row one gives."""
import math

import pytest

torch = pytest.importorskip("torch")

import dense_reference as ref  # noqa: E402
import dense_reference_rows as rows  # noqa: E402


@pytest.mark.parametrize("T,U", [(1.0, 0.05), (0.5, 2.0)])
def test_same_as_row_by_row(T, U):
    g = torch.Generator().manual_seed(0)
    R, V, k = 12, 37, 5
    z = torch.randn(R, V, generator=g)
    scores = torch.rand(R, k, generator=g)
    items = torch.randint(0, V, (R, k), generator=g)  # duplicates among them
    items[0] = -1
    scores[1] = -math.inf
    z[2] = -math.inf
    z[3, items[3]] = -math.inf
    z[4, ::3] = -math.inf
    items[5, 2], items[6, 0] = V, 1 << 40
    weight = torch.rand(R, generator=g)
    weight[7] = 0
    z[7, 3] = math.nan
    gl = torch.randn(R, generator=g)
    for a, b in zip(rows.distill(z, scores, items, weight, gl, T, U), ref.distill(z, scores, items, weight, gl, T, U)):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-14)
