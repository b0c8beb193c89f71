"""GPU tests of the dense operators where a block or a cluster works on many
rows or tiles: rings that are refilled and change phase, accumulators that are
handed back, rows taken over from clusters that have not started.

The sizes give every group of threads more rows than two rounds of its ring
(four slots at most), every pair of blocks more tiles than its two
accumulators, and every cluster more rows than the answers it has asked for,
on a GPU of 152 SMs.  Bounds as in test_gpu_dense.py.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import dense_reference as ref  # noqa: E402
import dense_reference_rows as rows_ref  # noqa: E402
from dense_reference import F64  # noqa: E402
from test_gpu_dense import (E, F8, HALVES, RMS_C, TYPES, _check_grad, _close, _linear_bound, _out, _randn,  # noqa: E402
                            _rms_grad_sizes, _strided)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_embedding_exact_gb300 as sec
    from sparse_embedding_exact_gb300 import build

    build.build()
    with sec.SparseCosine(1000, chunk_rows=256) as handle:
        yield handle


@pytest.fixture(autouse=True)
def _checked(h):
    yield
    h.check_device()


# ---------------------------------------------------------------- norm
# Groups of threads at a time are at most 152 x 4 blocks x 8 (256 columns of 16
# bits), x 2 (1001 columns, every row at another offset from 16 bytes); rows
# past 16,384 columns are taken by two blocks an SM.
RMS_SHAPES = [(50_000, 256), (13_000, 1001), (6000, 2056), (1000, 17_000), (700, 17_001)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", RMS_SHAPES)
def test_rms_norm_many_rows(h, dtype, rows, cols):
    x, w = _randn(rows, cols, dtype=dtype), _randn(cols, dtype=dtype, seed=1)
    r = _randn(rows, cols, std=2, dtype=dtype, seed=2)
    wy, ws, wr = ref.rms_norm(x, w, r)
    y, total, rstd = h.rms_norm(x, w, residual=r)
    _close(y, wy, _out(wy, dtype, RMS_C * E * wy.abs()), "y")
    _close(rstd, wr, RMS_C * E * wr, "rstd")
    _close(total, ws, _out(ws, dtype, E * ws.abs()), "total")
    q, scale, total8 = h.rms_norm_quantized(x, w, residual=r)
    assert torch.equal(total8, total)
    wscale = wy.abs().amax(1) / 448
    _close(scale, wscale, RMS_C * E * wscale, "scale")
    got = q.to(F64) * scale.to(F64)[:, None]
    _close(got, wy, (wy.abs() * 2.0 ** -4).maximum(wscale[:, None] * 2.0 ** -10) * (1 + 2.0 ** -10), "q")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(50_000, 256), (13_000, 1001)])
@pytest.mark.parametrize("pad,shift", [(3, 1), (8, 0)])
def test_rms_norm_many_rows_off_16_bytes(h, dtype, rows, cols, pad, shift):
    # both matrices at the same offsets, and at different ones
    x, w = _randn(rows, cols, dtype=dtype), _randn(cols, dtype=dtype, seed=1)
    r = _randn(rows, cols, std=2, dtype=dtype, seed=2)
    wy, ws, _ = ref.rms_norm(x, w, r)
    for a, b in ((_strided(x, pad, shift), _strided(r, pad, shift)), (x, _strided(r, pad, shift))):
        y, total, _ = h.rms_norm(a, w, residual=b)
        _close(y, wy, _out(wy, dtype, RMS_C * E * wy.abs()), "y")
        _close(total, ws, _out(ws, dtype, E * ws.abs()), "total")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", RMS_SHAPES)
def test_rms_norm_backward_many_rows(h, dtype, rows, cols):
    total, w = _randn(rows, cols, std=2, dtype=dtype), _randn(cols, dtype=dtype, seed=1)
    gy, gt = _randn(rows, cols, dtype=dtype, seed=2), _randn(rows, cols, dtype=dtype, seed=3)
    _, _, rstd = h.rms_norm(total, w)
    gx, gw = h.rms_norm_backward(gy, total, w, rstd, gt)
    wx, ww = ref.rms_norm_grad(gy, total, w, rstd, gt)
    size, wsize = _rms_grad_sizes(gy, total, w, rstd, gt)
    _close(gx, wx, _out(wx, dtype, RMS_C * E * size), "grad_x")
    _close(gw, ww, _out(ww, dtype, 4 * RMS_C * E * wsize), "grad_weight")
    again = h.rms_norm_backward(gy, total, w, rstd, gt)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)


# ---------------------------------------------------------------- linear
# 480 tiles of 256 x 256 for 76 pairs of blocks, of 2 to 16 stages; whole tiles'
# rows and columns, and ragged ones.
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,k,n", [(6000, 72, 5000), (6000, 1000, 5000), (6001, 1000, 5003)])
def test_linear_many_tiles(h, dtype, m, k, n):
    x, w = _randn(m, k, dtype=dtype), _randn(n, k, std=k ** -0.5, dtype=dtype, seed=1)
    b, r = _randn(n, seed=2), _randn(m, n, dtype=dtype, seed=3)
    y, pre = h.linear(x, w, bias=b, activation="silu", residual=r, save_pre=True)
    wy, wz, size = ref.linear(x, w, b, "silu", r)
    _close(pre, wz, _out(wz, dtype, _linear_bound(size, k)), "pre")
    _close(y, wy, _out(wy, dtype, _linear_bound(size, k) + 8 * E * (wy.abs() + r.to(F64).abs())), "y")
    again = h.linear(x, w, bias=b, activation="silu", residual=r, save_pre=True)
    assert torch.equal(again[0], y) and torch.equal(again[1], pre)


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("m,k,n", [(6000, 80, 5000), (6001, 1001, 5003)])
def test_linear_f8_many_tiles(h, out, m, k, n):
    x, w = _randn(m, k, std=100).to(F8), _randn(n, k, std=100, seed=1).to(F8)
    sx, sw = (_randn(m, seed=2).abs() + 0.01) / 1e4, (_randn(n, seed=3).abs() + 0.01) / k ** 0.5
    b, r = _randn(n, seed=4), _randn(m, n, dtype=out, seed=5)
    y = h.linear(x, w, bias=b, residual=r, x_scale=sx, w_scale=sw, out_dtype=out)
    wy, _, size = ref.linear(x, w, b, "none", r, sx, sw)
    _close(y, wy, _out(wy, out, _linear_bound(size, k) + 8 * E * (wy.abs() + r.to(F64).abs())), "y")


# grad_x of many tiles, grad_w of many tiles, and both with ragged edges.
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,k,n", [(5000, 4100, 264), (264, 4104, 5000), (3000, 4097, 2999)])
def test_linear_backward_many_tiles(h, dtype, m, k, n):
    x, w = _randn(m, k, dtype=dtype), _randn(n, k, std=k ** -0.5, dtype=dtype, seed=1)
    gy, pre = _randn(m, n, dtype=dtype, seed=2), _randn(m, n, dtype=dtype, seed=3)
    gx, gw, gb = h.linear_backward(gy, x, w, pre, "gelu")
    _check_grad(gx, gw, gb, gy, x, w, pre, "gelu", dtype)


# ---------------------------------------------------------------- distillation
def _case(R, V, k, dtype):
    """Logits, lists with duplicates and absent entries, weights: rows of every
    kind between each other."""
    g = torch.Generator(device="cuda").manual_seed(R + V)
    z = _randn(R, V, std=2.5, dtype=dtype)
    items = torch.randint(0, V, (R, k), device="cuda", generator=g)
    scores = torch.rand(R, k, device="cuda", generator=g)
    gone = torch.rand(R, k, device="cuda", generator=g) < 0.1
    kind = torch.randint(0, 12, (R,), device="cuda", generator=g)
    items = items.masked_fill(gone | (kind == 0)[:, None], -1)
    scores = scores.masked_fill((kind == 1)[:, None], -math.inf)
    z[kind == 2] = -math.inf                    # everything masked
    some = (kind == 3) | (kind == 4)
    z[some, ::3] = -math.inf
    weight = (torch.rand(R, device="cuda", generator=g) + 0.1).masked_fill((kind == 5) | (kind == 6), 0.0)
    z[kind == 5, 0] = math.nan                  # rows of weight 0 may hold anything
    return z, scores, items, weight, _randn(R, seed=8)


def _check_step(h, z, scores, items, weight, gl, T, U):
    kw = dict(weight=weight, temperature=T, teacher_temperature=U)
    loss, grad = h.distill_step(z, scores, items, gl, **kw)
    own = z.clone()
    loss2, grad2 = h.distill_step(own, scores, items, gl, in_place=True, **kw)
    assert grad2 is own and torch.equal(loss, loss2) and torch.equal(grad, own)
    del own, grad2
    wl, wg, terms, room = rows_ref.distill(z, scores, items, weight, gl, T, U)
    _close(loss, wl, 2.0 ** -19 * terms, "loss")
    _close(grad, wg, _out(wg, z.dtype, 2.0 ** -21 * room), "grad")


# Clusters of one block (10 rows each), of two and of four (many rows each; 304
# blocks run at a time).
@pytest.mark.parametrize("R,V,k,dtype", [(3000, 5000, 10, torch.bfloat16), (3000, 5001, 10, torch.float32),
                                         (1500, 60_000, 64, torch.bfloat16), (1500, 60_003, 7, torch.float16),
                                         (700, 100_000, 16, torch.float32), (700, 100_001, 256, torch.float32),
                                         (700, 200_001, 16, torch.bfloat16)])
def test_distill_step_many_rows(h, R, V, k, dtype):
    _check_step(h, *_case(R, V, k, dtype), 1.0, 0.1)


# Rows that eight blocks cannot hold, read twice.
@pytest.mark.parametrize("R,V,dtype", [(3, 250_001, torch.float32), (60, 300_000, torch.float32), (3, 500_003, torch.bfloat16),
                                       (60, 430_000, torch.float16)])
def test_distill_step_of_wide_rows_in_place(h, R, V, dtype):
    _check_step(h, *_case(R, V, 33, dtype), 0.5, 2.0)


# Loss alone and gradient alone over more rows than run at a time.
@pytest.mark.parametrize("R,V,dtype", [(3000, 5001, torch.float32), (1000, 60_000, torch.bfloat16)])
def test_distill_passes_many_rows(h, R, V, dtype):
    z, scores, items, weight, gl = _case(R, V, 10, dtype)
    kw = dict(weight=weight, temperature=2.0, teacher_temperature=0.1)
    loss, stats = h.distill(z, scores, items, **kw)
    grad = h.distill_backward(gl, z, scores, items, stats, **kw)
    wl, wg, terms, room = rows_ref.distill(z, scores, items, weight, gl, 2.0, 0.1)
    _close(loss, wl, 2.0 ** -19 * terms, "loss")
    _close(grad, wg, _out(wg, z.dtype, 2.0 ** -21 * room), "grad")
