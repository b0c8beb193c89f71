"""The 64-bit form of values kept in 8 bits: its bounds, exactness and edges; and
the calls' refusals that need no device."""
import math

import pytest

torch = pytest.importorskip("torch")

import kept_reference as ref  # noqa: E402
from dense_reference import F64  # noqa: E402


def _wide(rows, cols, dtype, seed=0):
    """Values over the type's whole range of exponents."""
    g = torch.Generator().manual_seed(seed)
    lo, hi = {torch.float32: (-140, 120), torch.bfloat16: (-130, 120), torch.float16: (-24, 15)}[dtype]
    e = torch.rand(rows, 1, generator=g) * (hi - lo) + lo
    return (torch.randn(rows, cols, generator=g).to(F64) * torch.exp2(e.to(F64))).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_error_and_exactness(dtype):
    x = _wide(300, 70, dtype)
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    q, e, v = ref.compressed(x)
    step = torch.exp2(e.to(F64) - 10).repeat_interleave(32, 1)[:, :70]
    assert ((v - x.to(F64)).abs() <= (x.to(F64).abs() * 2.0 ** -4).maximum(step)).all()
    inside = v.abs() <= ref.LARGEST[dtype]
    assert torch.equal(v[inside].to(dtype).to(F64), v[inside])  # exact in the type
    assert q.abs().max() <= 448
    assert torch.equal(q.to(torch.float32).to(torch.float8_e4m3fn).to(F64), q)  # e4m3's values
    big = ref._groups(q.abs()).amax(2)
    assert ((big > 208) | (e == ref.LEAST[dtype])).all()  # no smaller exponent would do


def test_by_torch():
    x = torch.randn(50, 96, generator=torch.Generator().manual_seed(3))
    q, e, _ = ref.compressed(x)
    scaled = x * torch.exp2(-e.float()).repeat_interleave(32, 1)
    assert torch.equal(scaled.to(torch.float8_e4m3fn).to(F64), q)


def test_edges():
    x = torch.zeros(4, 33)
    x[0, 0], x[0, 5] = 448.0, 1.0
    x[1, 0] = 449.0
    x[2, 3], x[2, 4], x[2, 5] = math.inf, math.nan, 3.0
    q, e, v = ref.compressed(x)
    assert e[0].tolist() == [0, -126] and e[1, 0] == 1 and v[0, 5] == 1
    assert torch.isnan(v[2, 3:5]).all() and v[2, 5] == 3 and e[2, 0] == -7
    assert not v[3].any() and (e[3] == -126).all()


def test_calls_without_a_handle_are_refused():
    from sparse_embedding_exact_gb300 import _abi, build

    build.build()
    lib, bad = _abi.load(), _abi.SS_ERR_INVALID_ARG
    assert lib.ss_compress(None, None, None, None) == bad
    assert lib.ss_expand(None, None, None, None) == bad
    assert lib.ss_linear_keep(None, None, None, None, None, None, 0, None, None, None, None, 0, None) == bad
    assert lib.ss_linear_kept_backward(None, None, None, None, None, None, None, 0, None, None, None, None, 0, None) == bad
    assert lib.ss_rms_norm_kept_backward(None, None, None, None, None, None, None, None, None, 0, None) == bad
    assert lib.ss_linear_keep_scratch(None, None, None) == 0
    assert lib.ss_linear_kept_backward_scratch(None, None, None, 0) == 0
    assert lib.ss_rms_norm_kept_backward_scratch(None, 5, 5, 0) == 0
