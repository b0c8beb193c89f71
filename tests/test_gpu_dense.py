"""GPU tests of the dense operators against their 64-bit forms.

Tolerances are bounds, not fits.  With u the output type's unit roundoff and
e = 2^-24: a value that is a few float32 operations and a sum of n terms of
size S is within u |value| + c e S of the exact one, c counting the roundings
along the longest chain of additions.
"""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import dense_reference as ref  # noqa: E402
from dense_reference import F64, ROUND, STEP  # noqa: E402

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
F8 = torch.float8_e4m3fn
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


@pytest.fixture(autouse=True)
def _checked(request):
    """No kernel of a test leaves a problem in the handle's status word."""
    yield
    if "h" in request.fixturenames and request.node.name != "test_distill_item_past_the_end":
        request.getfixturevalue("h").check_device()


def _randn(*shape, std=1.0, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def _strided(t, pad, shift=0):
    """The same matrix with `pad` more values a row, `shift` values into its buffer."""
    if pad == 0 and shift == 0:
        return t
    buf = torch.full((t.shape[0] * (t.shape[1] + pad) + shift + 16,), float("nan"), dtype=torch.float32,
                     device=t.device).to(t.dtype)
    v = buf.as_strided(t.shape, (t.shape[1] + pad, 1), shift)
    v.copy_(t)
    return v


def _close(got, want, bound, what=""):
    """|got - want| <= bound element by element, NaN and infinity where want has them."""
    got, want = got.to(F64), want.to(F64)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    same = fine | torch.isnan(want)
    assert torch.equal(got[~same], want[~same]), what
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: over the bound by {float(over.max())}"


def _out(want, dtype, extra):
    """Bound of an output: one rounding to its type, and the float32 error before it."""
    u = ROUND[dtype]
    return u * (want.to(F64).abs() + extra) + extra + STEP[dtype]


# ---------------------------------------------------------------- norm
# Longest chain: a thread's own additions (at most 64 in registers, 16384 / 1024
# vectors of 8 in the wide kernels) and two shuffle trees; the mean and its root
# halve it.  64 covers each.
RMS_C = 64

RMS_SHAPES = [(1, 1), (3, 7), (2, 128), (5, 1001), (300, 96), (700, 1024), (4, 4096), (3, 8191), (2, 16384), (2, 20000),
              (2, 33000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", RMS_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(h, dtype, rows, cols, residual):
    x, w = _randn(rows, cols, dtype=dtype), _randn(cols, dtype=dtype, seed=1)
    r = _randn(rows, cols, std=2, dtype=dtype, seed=2) if residual else None
    y, total, rstd = h.rms_norm(x, w, residual=r)
    wy, ws, wr = ref.rms_norm(x, w, r)
    _close(y, wy, _out(wy, dtype, RMS_C * E * wy.abs()), "y")
    _close(rstd, wr, RMS_C * E * wr, "rstd")
    if residual:
        _close(total, ws, _out(ws, dtype, E * ws.abs()), "total")
    else:
        assert total is x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", RMS_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_quantized(h, dtype, rows, cols, residual):
    x, w = _randn(rows, cols, dtype=dtype), _randn(cols, seed=1)  # float32 weights
    r = _randn(rows, cols, std=2, dtype=dtype, seed=2) if residual else None
    q, scale, total = h.rms_norm_quantized(x, w, residual=r)
    wy, ws, _ = ref.rms_norm(x, w, r)
    wscale = wy.abs().amax(1) / 448
    _close(scale, wscale, RMS_C * E * wscale, "scale")
    # half a step of e4m3: 2^-4 of the value, or 2^-10 below 2^-6
    got = q.to(F64) * scale.to(F64)[:, None]
    _close(got, wy, (wy.abs() * 2.0 ** -4).maximum(wscale[:, None] * 2.0 ** -10) * (1 + 2.0 ** -10), "y")
    assert (q.float().abs().amax(1) == 448).all()
    if residual:
        _close(total, ws, _out(ws, dtype, E * ws.abs()), "total")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_rms_norm_strides(h, dtype, pad, shift):
    x, w, r = _randn(9, 520, dtype=dtype), _randn(520, dtype=dtype, seed=1), _randn(9, 520, dtype=dtype, seed=2)
    y, total, rstd = h.rms_norm(_strided(x, pad, shift), w, residual=_strided(r, 2 * pad, shift))
    wy, ws, _ = ref.rms_norm(x, w, r)
    _close(y, wy, _out(wy, dtype, RMS_C * E * wy.abs()))
    _close(total, ws, _out(ws, dtype, E * ws.abs()))
    gx, gw = h.rms_norm_backward(_strided(x, pad, shift), _strided(total, pad), w, rstd, _strided(r, pad, shift))
    wx, ww = ref.rms_norm_grad(x, total, w, rstd, r)
    size, wsize = _rms_grad_sizes(x, total, w, rstd, r)
    _close(gx, wx, _out(wx, dtype, RMS_C * E * size))
    _close(gw, ww, _out(ww, dtype, RMS_C * E * wsize))


def _rms_grad_sizes(gy, total, w, rstd, gt):
    """What the gradient's sums add up, in absolute values."""
    a, _ = ref.rms_norm_grad(gy.abs(), torch.zeros_like(total), w.abs(), rstd, None if gt is None else gt.abs())
    xh = total.to(F64).abs() * rstd.to(F64)[:, None]
    g = gy.to(F64).abs() * w.to(F64).abs()
    return a + rstd.to(F64)[:, None] * xh * (g * xh).mean(1, keepdim=True), (gy.to(F64).abs() * xh).sum(0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", RMS_SHAPES + [(5000, 64), (1300, 2056)])
@pytest.mark.parametrize("past", [False, True])
def test_rms_norm_backward(h, dtype, rows, cols, past):
    total, w = _randn(rows, cols, std=2, dtype=dtype), _randn(cols, dtype=dtype, seed=1)
    gy = _randn(rows, cols, dtype=dtype, seed=2)
    gt = _randn(rows, cols, dtype=dtype, seed=3) if past else None
    _, _, rstd = h.rms_norm(total, w)
    gx, gw = h.rms_norm_backward(gy, total, w, rstd, gt)
    wx, ww = ref.rms_norm_grad(gy, total, w, rstd, gt)
    size, wsize = _rms_grad_sizes(gy, total, w, rstd, gt)
    _close(gx, wx, _out(wx, dtype, RMS_C * E * size), "grad_x")
    # rows in chains: a block's own (rows / 152 at most 64 here), then the blocks' in eights
    _close(gw, ww, _out(ww, dtype, 4 * RMS_C * E * wsize), "grad_weight")
    again = h.rms_norm_backward(gy, total, w, rstd, gt)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)


def test_rms_norm_gradient_by_differences(h):
    # A step of 2^-4 along a direction d changes f = sum(gy y) by h <grad, d> +
    # O(h^3); f of the 64-bit form at the same points, the gradient the kernel's.
    x, w, gy = _randn(6, 200), _randn(200, seed=1), _randn(6, 200, seed=2)
    y, total, rstd = h.rms_norm(x, w)
    gx, gw = h.rms_norm_backward(gy, total, w, rstd)
    for at, grad, f in ((x, gx, lambda v: ref.rms_norm(v, w)[0]), (w, gw, lambda v: ref.rms_norm(x, v)[0])):
        d = _randn(*at.shape, seed=5).to(F64)
        s = 2.0 ** -10
        up, down = ((gy.to(F64) * f(at.to(F64) + k * s * d)).sum() for k in (1, -1))
        slope = float((grad.to(F64) * d).sum())
        assert abs(float(up - down) / (2 * s) - slope) <= 1e-5 * float((grad.to(F64) * d).abs().sum()) + 1e-5


@pytest.mark.parametrize("dtype", TYPES)
def test_rms_norm_special_rows(h, dtype):
    x = _randn(6, 256, dtype=dtype)
    x[0] = 0
    x[1] = torch.finfo(dtype).tiny
    x[2, 5] = math.inf
    x[3, 7] = math.nan
    x[4] = 0
    x[4, 9] = 1
    w = torch.ones(256, device="cuda")
    y, _, rstd = h.rms_norm(x, w)
    wy, _, wr = ref.rms_norm(x, w)
    _close(y, wy, _out(wy, dtype, RMS_C * E * wy.abs()))
    _close(rstd, wr, RMS_C * E * wr)
    q, scale, _ = h.rms_norm_quantized(x, w)
    assert not q[0].float().any() and float(scale[0]) == 0
    assert torch.isnan(q[2, 5].float()) and not q[2, :5].float().any() and torch.isnan(scale[2])
    assert torch.isnan(q[3].float()).all() and torch.isnan(scale[3])
    assert float(q[4, 9].float()) == 448 and float(q[4].float().sum()) == 448
    tiny = q[1].to(F64) * scale[1].to(F64)
    _close(tiny, wy[1], wy[1].abs() * 2.0 ** -4 + STEP[torch.float32] * 448)


def test_rms_norm_no_rows(h):
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    y, total, rstd = h.rms_norm(x, w, residual=x)
    assert y.shape == (0, 64) and rstd.numel() == 0
    gx, gw = h.rms_norm_backward(x, x, w, rstd)
    assert gx.shape == (0, 64) and not gw.any()


# ---------------------------------------------------------------- linear
def _linear_bound(size, k):
    """The products are exact; a partial sum of size S is rounded (or cut) to
    float32 once for each 16 of them, the tree within them and the cluster's
    eight shares: at most 2^-23 S each; then scale, bias and activation (whose
    slopes stay below 1.2)."""
    return 1.2 * (k / 16 + 32) * 2.0 ** -23 * size


LINEAR_SHAPES = [(1, 64, 64), (1, 1001, 777), (2, 512, 1000), (3, 33, 5), (4, 4096, 257), (5, 64, 64), (7, 100, 300),
                 (16, 4096, 512), (33, 1024, 129), (64, 72, 4096), (130, 640, 200), (257, 128, 256), (300, 1000, 1000),
                 (1000, 2048, 520), (129, 16, 130), (2100, 264, 2056)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,k,n", LINEAR_SHAPES)
def test_linear(h, dtype, m, k, n):
    x, w = _randn(m, k, dtype=dtype), _randn(n, k, std=k ** -0.5, dtype=dtype, seed=1)
    b, r = _randn(n, seed=2), _randn(m, n, dtype=dtype, seed=3)
    y, pre = h.linear(x, w, bias=b, activation="gelu", residual=r, save_pre=True)
    wy, wz, size = ref.linear(x, w, b, "gelu", r)
    _close(pre, wz, _out(wz, dtype, _linear_bound(size, k)), "pre")
    _close(y, wy, _out(wy, dtype, _linear_bound(size, k) + 8 * E * (wy.abs() + r.to(F64).abs())), "y")
    plain = h.linear(x, w, out_dtype=torch.float32)
    wy, _, size = ref.linear(x, w)
    _close(plain, wy, _out(wy, torch.float32, _linear_bound(size, k)), "plain")
    assert torch.equal(plain, h.linear(x, w, out_dtype=torch.float32))


@pytest.mark.parametrize("m,k,n", LINEAR_SHAPES)
@pytest.mark.parametrize("out", TYPES)
def test_linear_f8(h, m, k, n, out):
    x, w = _randn(m, k, std=100).to(F8), _randn(n, k, std=100, seed=1).to(F8)
    sx, sw = _randn(m, seed=2).abs() + 0.01, _randn(n, seed=3).abs() + 0.01
    sx, sw = sx / 1e4, sw / k ** 0.5
    b, r = _randn(n, seed=4), _randn(m, n, dtype=out, seed=5)
    y = h.linear(x, w, bias=b, activation="silu", residual=r, x_scale=sx, w_scale=sw, out_dtype=out)
    wy, _, size = ref.linear(x, w, b, "silu", r, sx, sw)
    _close(y, wy, _out(wy, out, _linear_bound(size, k) + 8 * E * (wy.abs() + r.to(F64).abs())))


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu", "log1p_relu"])
@pytest.mark.parametrize("m", [3, 40, 400])
def test_linear_activations(h, name, m):
    k, n, dtype = 64, 136, torch.bfloat16
    x, w = _randn(m, k, std=3, dtype=dtype), _randn(n, k, dtype=dtype, seed=1)  # |z| up to 100
    y, pre = h.linear(x, w, activation=name, out_dtype=torch.float32, save_pre=True)
    wy, wz, size = ref.linear(x, w, None, name)
    _close(y, wy, _out(wy, torch.float32, _linear_bound(size, k) + 16 * E * (wz.abs() + 1)), "y")
    gy = _randn(m, n, dtype=dtype, seed=2)
    pre = wz.to(dtype)
    gx, gw, gb = h.linear_backward(gy, x, w, pre, name, grad_dtype=torch.float32)
    _check_grad(gx, gw, gb, gy, x, w, pre, name, torch.float32)


def _check_grad(gx, gw, gb, gy, x, w, pre, name, dtype):
    wx, ww, wb, gz = ref.linear_grad(gy, x, w, pre, name)
    # gz enters the products rounded to 16 bits; the slope's own float32 error
    # is 2^-20 of its largest value 1.2 (relative to grad_y)
    u = 0.0 if name == "none" else ROUND[x.dtype]
    off = gz.abs() * u + 2.0 ** -20 * 1.2 * gy.to(F64).abs() + (STEP[x.dtype] if u else 0)
    size = gz.abs() + off
    M, N = gz.shape
    _close(gx, wx, _out(wx, dtype, off @ w.to(F64).abs() + _linear_bound(size @ w.to(F64).abs(), N)), "grad_x")
    _close(gw, ww, _out(ww, dtype, off.t() @ x.to(F64).abs() + _linear_bound(size.t() @ x.to(F64).abs(), M)), "grad_w")
    own = (2.0 ** -20 * 1.2 * gy.to(F64).abs()).sum(0) if name != "none" else 0
    _close(gb, wb, own + (64 + M / 8) * E * gz.abs().sum(0), "grad_bias")


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", ["none", "gelu"])
@pytest.mark.parametrize("m,k,n", LINEAR_SHAPES)
def test_linear_backward(h, dtype, name, m, k, n):
    x, w = _randn(m, k, dtype=dtype), _randn(n, k, std=k ** -0.5, dtype=dtype, seed=1)
    gy, pre = _randn(m, n, dtype=dtype, seed=2), _randn(m, n, dtype=dtype, seed=3)
    gx, gw, gb = h.linear_backward(gy, x, w, pre if name != "none" else None, name)
    _check_grad(gx, gw, gb, gy, x, w, pre, name, dtype)
    again = h.linear_backward(gy, x, w, pre if name != "none" else None, name)
    assert all(torch.equal(a, b) for a, b in zip(again, (gx, gw, gb)))


@pytest.mark.parametrize("m", [2, 30, 300])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_linear_strides(h, m, pad, shift):
    k, n, dtype = 136, 264, torch.float16
    x, w = _randn(m, k, dtype=dtype), _randn(n, k, std=k ** -0.5, dtype=dtype, seed=1)
    r, gy = _randn(m, n, dtype=dtype, seed=2), _randn(m, n, dtype=dtype, seed=3)
    xs, ws, rs, gs = (_strided(t, pad, shift) for t in (x, w, r, gy))
    y = h.linear(xs, ws, residual=rs)
    wy, _, size = ref.linear(x, w, None, "none", r)
    _close(y, wy, _out(wy, dtype, _linear_bound(size, k) + 8 * E * (wy.abs() + r.to(F64).abs())))
    for name in ("none", "silu"):
        gx, gw, gb = h.linear_backward(gs, xs, ws, rs, name)
        _check_grad(gx, gw, gb, gy, x, w, r, name, dtype)


def test_linear_gradient_by_differences(h):
    m, k, n, dtype = 40, 24, 72, torch.bfloat16
    x, w, gy = _randn(m, k, dtype=dtype), _randn(n, k, dtype=dtype, seed=1), _randn(m, n, dtype=dtype, seed=2)
    b = _randn(n, seed=3)
    _, pre = h.linear(x, w, bias=b, activation="silu", save_pre=True)
    gx, gw, gb = h.linear_backward(gy, x, w, pre, "silu", grad_dtype=torch.float32)
    f = {0: lambda v: ref.linear(v, w, b, "silu")[0], 1: lambda v: ref.linear(x, v, b, "silu")[0],
         2: lambda v: ref.linear(x, w, v, "silu")[0]}
    for i, (at, grad) in enumerate(((x, gx), (w, gw), (b, gb))):
        d, s = _randn(*at.shape, seed=5).to(F64), 2.0 ** -10
        up, down = ((gy.to(F64) * f[i](at.to(F64) + q * s * d)).sum() for q in (1, -1))
        # the kept z and gz are rounded to 8 bits: 2^-8 of each term, twice
        room = 2 * ROUND[dtype] * float((gy.to(F64).abs() @ w.to(F64).abs()).sum() + gy.to(F64).abs().sum() * 24)
        assert abs(float(up - down) / (2 * s) - float((grad.to(F64) * d).sum())) <= 0.02 * room


@pytest.mark.parametrize("m", [1, 8, 200])
def test_linear_special_values(h, m):
    dtype, k, n = torch.bfloat16, 64, 96
    x, w = _randn(m, k, dtype=dtype), _randn(n, k, dtype=dtype, seed=1)
    x[0, 3], w[7, 5] = math.nan, math.inf
    y = h.linear(x, w, activation="relu")
    wy = ref.linear(x, w, None, "none")[0]
    wy = torch.where(torch.isnan(wy), wy, torch.clamp_min(wy, 0))
    assert torch.equal(torch.isnan(y), torch.isnan(wy)) and torch.equal(torch.isinf(y), torch.isinf(wy))


@pytest.mark.parametrize("m", [0, 1, 5, 300])
def test_linear_empty(h, m):
    dtype = torch.float16
    x, w, b = torch.empty(m, 0, dtype=dtype, device="cuda"), torch.empty(40, 0, dtype=dtype, device="cuda"), _randn(40)
    y = h.linear(x, w, bias=b, activation="relu")
    assert torch.equal(y, torch.relu(b).to(dtype).expand(m, 40))
    gx, gw, gb = h.linear_backward(y, x, w)
    assert gx.shape == (m, 0) and gw.shape == (40, 0)
    assert (gb - y.float().sum(0)).abs().max() <= 1e-3 * max(1, m)
    x, w = _randn(m, 24, dtype=dtype), torch.empty(0, 24, dtype=dtype, device="cuda")
    assert h.linear(x, w).shape == (m, 0)
    gx, gw, gb = h.linear_backward(torch.empty(m, 0, dtype=dtype, device="cuda"), x, w)
    assert not gx.any() and gw.shape == (0, 24) and gb.numel() == 0


# ---------------------------------------------------------------- distillation
def _lists(R, V, k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    items = torch.stack([torch.randperm(max(V, k), device="cuda", generator=g)[:k] for _ in range(R)])
    scores = torch.rand(R, k, device="cuda", generator=g).sort(1, descending=True).values
    gone = (items >= V) | (torch.rand(R, k, device="cuda", generator=g) < 0.1)
    return scores.masked_fill(gone, -math.inf), items.masked_fill(gone, -1)


def _check_distill(h, z, scores, items, weight, gl, T, U):
    loss, stats = h.distill(z, scores, items, weight=weight, temperature=T, teacher_temperature=U)
    grad = h.distill_backward(gl, z, scores, items, stats, weight=weight, temperature=T, teacher_temperature=U)
    wl, wg, terms, room = ref.distill(z, scores, items, weight, gl, T, U)
    # each exponential is within (|argument| + 16) 2^-22 of itself (the argument
    # rounded twice, the instruction's 2^-22), and so are the sums of them
    _close(loss, wl, 2.0 ** -19 * terms, "loss")
    _close(grad, wg, _out(wg, z.dtype, 2.0 ** -21 * room), "grad")
    step_loss, step_grad = h.distill_step(z, scores, items, gl, weight=weight, temperature=T, teacher_temperature=U)
    _close(step_loss, wl, 2.0 ** -19 * terms, "step loss")
    _close(step_grad, wg, _out(wg, z.dtype, 2.0 ** -21 * room), "step grad")
    return loss, grad


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V,k", [(1, 1, 1), (2, 7, 3), (3, 33, 10), (5, 1000, 64), (300, 501, 2), (2, 4099, 256),
                                   (3, 70001, 33), (1, 200000, 64), (2, 500003, 5), (40, 30000, 10)])
@pytest.mark.parametrize("T,U", [(1.0, 0.05), (0.5, 2.0)])
def test_distill(h, dtype, R, V, k, T, U):
    z = _randn(R, V, std=2.5, dtype=dtype)
    scores, items = _lists(R, V, k)
    weight = (_randn(R, seed=7).abs() + 0.1).masked_fill(torch.arange(R, device="cuda") % 3 == 2, 0.0)
    gl = _randn(R, seed=8)
    a = _check_distill(h, z, scores, items, weight, gl, T, U)
    b = _check_distill(h, z, scores, items, weight, gl, T, U)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [64, 1003, 50001])
def test_distill_masks(h, dtype, V):
    z = _randn(8, V, std=2, dtype=dtype)
    scores, items = _lists(8, V, 12)
    items[0] = -1                        # no entry
    scores[1] = -math.inf                # no entry
    z[2] = -math.inf                     # everything masked
    z[3, items[3].clamp_min(0)] = -math.inf  # every listed item masked
    z[4, ::3] = -math.inf
    low = torch.finfo(dtype).min         # masks of the type's lowest value
    z[5] = torch.where(torch.arange(V, device="cuda") % 2 == 0, z[5], torch.full_like(z[5], low))
    items[5] = torch.where(items[5] % 2 == 0, items[5], torch.full_like(items[5], -1))
    z[6] = low                           # nothing but the lowest value: all equal
    weight = torch.ones(8, device="cuda")
    weight[7] = 0
    z[7, 0] = math.nan                   # a padding row may hold anything
    loss, grad = _check_distill(h, z, scores, items, weight, None, 1.0, 0.1)
    assert not loss[[0, 1, 2, 3, 7]].any() and not grad[[0, 1, 2, 3, 7]].any()


def test_distill_nan_and_infinity(h):
    z = _randn(4, 5000)
    scores, items = _lists(4, 5000, 6)
    z[1, 17], z[2, 19] = math.nan, math.inf
    scores[3, 0], items[3, 0] = math.nan, 11
    for loss, grad in (h.distill_step(z, scores, items),
                       (lambda f: (f[0], h.distill_backward(None, z, scores, items, f[1])))(h.distill(z, scores, items))):
        assert torch.isfinite(loss[0]) and torch.isfinite(grad[0]).all()
        assert torch.isnan(loss[1:]).all()
        assert torch.isnan(grad[1]).all() and torch.isnan(grad[2, 19]) and torch.isnan(grad[3, 11])


@pytest.mark.parametrize("dtype", TYPES)
def test_distill_duplicates_and_ends(h, dtype):
    z = _randn(2, 4097, dtype=dtype)
    items = torch.tensor([[0, 4096, 5, 5, 5], [4096, 4096, 0, 0, 2048]], device="cuda")
    scores = torch.rand(2, 5, device="cuda")
    _check_distill(h, z, scores, items, None, None, 1.0, 1.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_distill_strides(h, dtype, pad, shift):
    z = _strided(_randn(5, 30001, dtype=dtype), pad, shift)
    scores, items = _lists(5, 30001, 9)
    _check_distill(h, z, scores, items, None, None, 1.0, 0.2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V", [(3, 1000), (2, 200001), (400, 5000)])
def test_distill_in_place(h, dtype, R, V):
    z = _randn(R, V, dtype=dtype)
    z[0, ::5] = -math.inf
    scores, items = _lists(R, V, 16)
    loss, grad = h.distill_step(z, scores, items, temperature=2.0, teacher_temperature=0.1)
    own = z.clone()
    loss2, grad2 = h.distill_step(own, scores, items, temperature=2.0, teacher_temperature=0.1, in_place=True)
    assert grad2 is own and torch.equal(grad, own) and torch.equal(loss, loss2)


def test_distill_gradient_by_differences(h):
    z = _randn(3, 400)
    scores, items = _lists(3, 400, 8)
    gl = _randn(3, seed=4)
    _, grad = h.distill_step(z, scores, items, gl, temperature=1.5, teacher_temperature=0.3)
    d, s = _randn(3, 400, seed=5).to(F64), 2.0 ** -10
    up, down = ((ref.distill(z.to(F64) + k * s * d, scores, items, None, None, 1.5, 0.3)[0] * gl.to(F64)).sum()
                for k in (1, -1))
    slope = float((grad.to(F64) * d).sum())
    assert abs(float(up - down) / (2 * s) - slope) <= 1e-5 * float((grad.to(F64) * d).abs().sum()) + 1e-5


def test_distill_no_rows_and_no_items(h):
    z = torch.empty(0, 10, device="cuda")
    s, i = torch.empty(0, 3, device="cuda"), torch.empty(0, 3, dtype=torch.int64, device="cuda")
    loss, grad = h.distill_step(z, s, i)
    assert loss.numel() == 0 and grad.shape == (0, 10)
    z = torch.empty(2, 0, device="cuda")
    loss, grad = h.distill_step(z, torch.zeros(2, 3, device="cuda"),
                                torch.full((2, 3), -1, dtype=torch.int64, device="cuda"))
    assert not loss.any() and grad.shape == (2, 0)


def test_distill_item_past_the_end(h):
    import sparse_embedding_exact_gb300 as sec

    z = _randn(2, 100)
    items = torch.tensor([[3, 100], [1 << 40, 5]], device="cuda")
    scores = torch.tensor([[0.5, 0.4], [0.3, 0.2]], device="cuda")
    loss, grad = h.distill_step(z, scores, items)
    wl, wg, _, room = ref.distill(z, scores, items)
    _close(grad, wg, _out(wg, z.dtype, 2.0 ** -21 * room))
    with pytest.raises(sec.SparseCosError) as err:
        h.check_device()
    assert err.value.status == sec._abi.SS_ERR_OUT_OF_RANGE
    h.check_device()


# ---------------------------------------------------------------- all of them
def test_offsets_past_32_bits(h):
    # two rows further apart than 2^32 bytes and 2^31 values
    far, dtype = (1 << 31) + 8, torch.bfloat16
    buf = torch.empty(far + 4096, dtype=dtype, device="cuda")
    x = buf.as_strided((2, 1024), (far, 1))
    x.copy_(_randn(2, 1024, dtype=dtype))
    near = x.contiguous()
    w = _randn(1024, dtype=dtype, seed=1)
    for a, b in zip(h.rms_norm(x, w, residual=x), h.rms_norm(near, w, residual=near)):
        assert torch.equal(a, b)
    _, _, rstd = h.rms_norm(near, w)
    assert all(torch.equal(a, b) for a, b in zip(h.rms_norm_backward(x, x, w, rstd), h.rms_norm_backward(near, near, w, rstd)))
    scores, items = _lists(2, 1024, 5)
    for a, b in zip(h.distill_step(x, scores, items), h.distill_step(near, scores, items)):
        assert torch.equal(a, b)
    wide = _randn(600, 1024, dtype=dtype, seed=2)
    assert torch.equal(h.linear(x, wide), h.linear(near, wide))
    assert torch.equal(h.linear(wide, x), h.linear(wide, near))


def test_another_stream(h):
    s = torch.cuda.Stream()
    x, w = _randn(300, 512, dtype=torch.bfloat16), _randn(640, 512, std=0.05, dtype=torch.bfloat16, seed=1)
    g, k = _randn(512, dtype=torch.bfloat16, seed=2), _lists(300, 640, 7)

    def layer(stream):
        y, total, rstd = h.rms_norm(x, g, residual=x, stream=stream)
        z, pre = h.linear(y, w, activation="silu", save_pre=True, stream=stream)
        loss, grad = h.distill_step(z, *k, stream=stream)
        gx, gw, gb = h.linear_backward(grad, y, w, pre, "silu", stream=stream)
        return (loss, gw, gb) + h.rms_norm_backward(gx, total, g, rstd, stream=stream)

    want = layer(None)
    s.wait_stream(torch.cuda.current_stream())
    got = layer(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # and as a graph
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = layer(None)
    for t in kept:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, kept))


def test_refusals(h):
    import sparse_embedding_exact_gb300 as sec

    bf, f16 = torch.bfloat16, torch.float16
    x, w = _randn(8, 64, dtype=bf), _randn(32, 64, dtype=bf)
    g = torch.ones(64, device="cuda")
    scores, items = _lists(8, 64, 4)

    def refused(status, call, *args, **kw):
        before = h.kernel_launches()
        with pytest.raises(sec.SparseCosError) as err:
            call(*args, **kw)
        assert err.value.status == status and h.kernel_launches() == before

    bad, limit = sec._abi.SS_ERR_INVALID_ARG, sec._abi.SS_ERR_LIMIT
    refused(bad, h.rms_norm, x, g[:32].contiguous())
    refused(bad, h.rms_norm, x, g.to(f16))
    refused(bad, h.rms_norm, x, g, residual=x.to(f16))
    refused(bad, h.rms_norm, x, g, residual=x[:4])
    refused(bad, h.rms_norm, x, g, eps=-1.0)
    refused(bad, h.rms_norm, x, g, eps=math.nan)
    refused(bad, h.rms_norm, x.to(F8), g)
    refused(bad, h.rms_norm, x[:, :0], g[:0])
    refused(bad, h.rms_norm_backward, x.to(f16), x, g, torch.ones(8, device="cuda"))
    refused(bad, h.linear, x, w[:, :32])
    refused(bad, h.linear, x, w.to(f16))
    refused(bad, h.linear, x.float(), w.float())
    refused(bad, h.linear, x, w, out_dtype=f16)
    refused(bad, h.linear, x, w, residual=x)
    refused(bad, h.linear, x.to(F8), w.to(F8))
    refused(bad, h.linear, x, w, x_scale=torch.ones(8, device="cuda"), w_scale=torch.ones(32, device="cuda"))
    refused(bad, h.linear_backward, x[:, :32], x, w, None, "gelu")
    refused(bad, h.linear_backward, x, x, w)
    refused(bad, h.distill, x, scores, items, temperature=0.0)
    refused(bad, h.distill, x, scores, items, temperature=math.inf)
    refused(bad, h.distill, x.to(F8), scores, items)
    refused(limit, h.distill, x, torch.zeros(8, 257, device="cuda"), torch.zeros(8, 257, dtype=torch.int64, device="cuda"))
    refused(limit, h.distill, x, torch.zeros(8, 0, device="cuda"), torch.zeros(8, 0, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        h.linear(x, w, activation="swish")
    with pytest.raises(ValueError):
        h.linear(x.cpu(), w)
    with pytest.raises(ValueError):
        h.linear(x.t(), w)
    with pytest.raises(ValueError):
        h.linear(x, w, bias=torch.ones(31, device="cuda"))
    with pytest.raises(TypeError):
        h.linear(x, w, bias=torch.ones(32, device="cuda", dtype=bf))
    with pytest.raises(TypeError):
        h.distill(x, scores, items.int())
    with pytest.raises(ValueError):
        h.distill(x, scores[:4], items)
    # the C calls check their own scratch and places
    lib, a = h._lib, sec._abi
    odd = _randn(8, 65, dtype=bf)[:, :63]
    code = {torch.float32: a.SS_VALUES_F32, bf: a.SS_VALUES_BF16}

    def record(t):
        rows = t.shape[0] if t.dim() == 2 else 1
        return a.ss_dense(t.data_ptr(), rows, t.shape[-1], t.stride(0) if rows > 1 else t.shape[-1], code[t.dtype])

    ref_of = ctypes.addressof
    keep = [record(t) for t in (odd, _randn(32, 63, dtype=bf), torch.empty(8, 32, dtype=bf, device="cuda"), x, g, g[:63])]
    m = [ref_of(t) for t in keep]
    assert lib.ss_linear_scratch(h._h, m[0], m[1]) > 0
    assert lib.ss_linear(h._h, m[0], None, m[1], None, None, 0, None, None, m[2], None, 0, None) == a.SS_ERR_INVALID_ARG
    z = m[3]
    assert lib.ss_distill_backward(h._h, None, z, scores.data_ptr(), items.data_ptr(), 4, 1.0, 1.0, None,
                                   scores.data_ptr(), z, None) == a.SS_ERR_INVALID_ARG
    low = a.ss_dense(x.data_ptr(), 8, 64, 63, a.SS_VALUES_BF16)
    assert lib.ss_rms_norm(h._h, ref_of(low), None, m[4], 1e-6, None, z, None, None, None) == a.SS_ERR_INVALID_ARG
    off = a.ss_dense(x.data_ptr() + 1, 8, 63, 64, a.SS_VALUES_BF16)
    assert lib.ss_rms_norm(h._h, ref_of(off), None, m[5], 1e-6, None, ref_of(off), None, None, None) == a.SS_ERR_INVALID_ARG
