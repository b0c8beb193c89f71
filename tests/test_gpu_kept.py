"""GPU tests of activations kept in 8 bits: codes and scales bit for bit against
the 64-bit form, the gradients from them against the formulas of the values
that they stand for."""
import math

import pytest

torch = pytest.importorskip("torch")

import dense_reference as dense  # noqa: E402
import kept_reference as ref  # noqa: E402
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


def _strided(t, pad, shift=0):
    buf = torch.zeros((t.shape[0] * (t.shape[1] + pad) + shift + 16,), dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device=t.device)
    v = buf.view(t.dtype).as_strided(t.shape, (t.shape[1] + pad, 1), shift)
    v.copy_(t)
    return v


def _close(got, want, bound, what=""):
    """|got - want| <= bound element by element, NaN where want has it."""
    got, want = got.to(F64), want.to(F64)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: over the bound by {float(over.max())}"


def _out(want, dtype, extra):
    u = ROUND[dtype]
    return u * (want.to(F64).abs() + extra) + extra + STEP[dtype]


def _same_codes(codes, scale, x, cols=None):
    """codes and scales are the 64-bit form's, and expand what they stand for."""
    q, e, _ = ref.compressed(x)
    assert codes.dtype == torch.float8_e4m3fn and scale.dtype == torch.float8_e8m0fnu
    assert codes.shape == x.shape and scale.shape == e.shape
    assert torch.equal(ref.exponents_of(scale), e)
    got = codes.to(F64)
    assert torch.equal(torch.isnan(got), torch.isnan(q))
    assert torch.equal(got.nan_to_num(0.0), q.nan_to_num(0.0))


SHAPES = [(1, 1), (1, 32), (3, 7), (2, 33), (5, 64), (4, 4096), (300, 96), (70, 1001), (33, 8), (1000, 24), (3, 20_008), (9, 255)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_compress(h, dtype, rows, cols):
    x = _randn(rows, cols, std=3.0)
    x = x * torch.exp2(torch.randint(-30, 30, (rows, 1), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).float() / 3)
    x = x.to(dtype)
    codes, scale = h.compress(x)
    _same_codes(codes, scale, x)
    for out in TYPES:
        y = h.expand(codes, scale, out)
        assert y.dtype == out and torch.equal(y.to(F64), ref.stand_for(codes, scale, out).to(out).to(F64))
    flat, fscale = h.compress(x[0])
    assert flat.shape == (cols,) and torch.equal(flat.view(torch.uint8), codes[0].view(torch.uint8))
    assert torch.equal(h.expand(flat, fscale, dtype), h.expand(codes, scale, dtype)[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_compress_strides(h, dtype, pad, shift):
    x = _randn(37, 200, dtype=dtype)
    codes, scale = h.compress(_strided(x, pad, shift))
    _same_codes(codes, scale, x)
    y = h.expand(_strided(codes, pad, shift), scale, dtype)
    assert torch.equal(y.to(F64), ref.stand_for(codes, scale))


@pytest.mark.parametrize("dtype", TYPES)
def test_compress_edges(h, dtype):
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x = torch.zeros(12, 70, device="cuda")
    x[0, 0], x[0, 40], x[0, 69] = 448, 1.0, -1.75
    x[1, 0], x[1, 1] = 449.0, -0.0
    x[2, 3], x[2, 4], x[2, 5], x[2, 6] = math.inf, math.nan, 3.0, -math.inf
    x[3] = math.inf
    x[4] = math.nan
    x = x.to(dtype)
    x[5], x[6] = big, -big
    x[7] = tiny
    x[8, ::2] = tiny * 2.0 ** -5
    x[9] = _randn(70, seed=2).to(dtype) * tiny
    x[10] = (1 + torch.arange(70, device="cuda") / 16).to(dtype)  # ties
    codes, scale = h.compress(x)
    _same_codes(codes, scale, x)
    y = h.expand(codes, scale, dtype)
    want = ref.stand_for(codes, scale, dtype)
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(y.to(F64).nan_to_num(0.0), want.nan_to_num(0.0))
    assert torch.isfinite(y[5:7]).all()


def test_scales_of_any_byte(h):
    scale = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].view(torch.float8_e8m0fnu)
    codes = _randn(256, 32, std=100.0).to(torch.float8_e4m3fn)
    y = h.expand(codes, scale, torch.float32)
    want = ref.stand_for(codes, scale, torch.float32).to(torch.float32)
    assert torch.isnan(y[255]).all() and torch.equal(y[:255], want[:255])


def test_empty(h):
    for shape in ((0, 40), (3, 0), (0, 0)):
        codes, scale = h.compress(torch.empty(shape, device="cuda", dtype=torch.bfloat16))
        assert codes.shape == shape and h.expand(codes, scale).shape == shape


# ---------------------------------------------------------------- linear layers
LAYERS = [(1, 64, 32), (2, 512, 1000), (3, 33, 5), (5, 64, 64), (16, 4096, 512), (33, 1024, 129), (130, 640, 200), (257, 128, 256),
          (300, 1000, 1000), (1000, 2048, 520), (129, 16, 130), (1, 1001, 777), (2100, 264, 2056)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,k,n", LAYERS)
def test_linear_keeps(h, dtype, m, k, n):
    x, w = _randn(m, k, dtype=dtype), _randn(n, k, std=k ** -0.5, dtype=dtype, seed=1)
    b, r = _randn(n, seed=2), _randn(m, n, dtype=dtype, seed=3)
    y, pre, scale = h.linear(x, w, bias=b, activation="gelu", residual=r, compress_pre=True)
    wy, wz, size = dense.linear(x, w, b, "gelu", r)
    room = 1.2 * (k / 16 + 32) * 2.0 ** -23 * size  # the float32 sums, as in the layer's own tests
    _close(y, wy, _out(wy, dtype, room + 8 * E * (wy.abs() + r.to(F64).abs())), "y")
    assert pre.shape == (m, n) and scale.shape == (m, (n + 31) // 32)
    e = ref.exponents_of(scale)
    # the exponents of z, or where the sums' error reaches across a border the next
    low, high = (ref.exponents(torch.clamp_min(wz.abs() + q * room, 0), ref.LEAST[dtype]) for q in (-1, 1))
    assert ((e >= low) & (e <= high)).all()
    step = torch.exp2(e.to(F64) - 10).repeat_interleave(32, 1)[:, :n]
    _close(ref.stand_for(pre, scale), wz, (wz.abs() * 2.0 ** -4).maximum(step) * (1 + 2.0 ** -10) + 2 * room, "pre")
    # z in float32, compressed in a call of its own, has the same codes where
    # the sums are cut alike
    _, z = h.linear(x, w, bias=b, out_dtype=torch.float32, save_pre=True)
    differ = (h.compress(z)[0].to(F64) - pre.to(F64)).abs() > 0
    assert float(differ.double().mean()) <= 0.02


def test_linear_keeps_from_8_bits(h):
    m, k, n = 70, 256, 160
    x, w = _randn(m, k, std=100).to(torch.float8_e4m3fn), _randn(n, k, std=100, seed=1).to(torch.float8_e4m3fn)
    sx, sw = (_randn(m, seed=2).abs() + 0.01) / 1e4, (_randn(n, seed=3).abs() + 0.01) / k ** 0.5
    y, pre, scale = h.linear(x, w, activation="silu", x_scale=sx, w_scale=sw, compress_pre=True)
    wy, wz, size = dense.linear(x, w, None, "silu", None, sx, sw)
    room = 1.2 * (k / 16 + 32) * 2.0 ** -23 * size
    _close(y, wy, _out(wy, torch.bfloat16, room + 8 * E * wy.abs()), "y")
    step = torch.exp2(ref.exponents_of(scale).to(F64) - 10).repeat_interleave(32, 1)[:, :n]
    _close(ref.stand_for(pre, scale), wz, (wz.abs() * 2.0 ** -4).maximum(step) * (1 + 2.0 ** -10) + 2 * room, "pre")


def _check_layer(grads, gy, x, w, pre, name, dtype):
    """Against the gradients of the values x and pre (64 bits)."""
    gz = gy.to(F64) * dense.act_grad(pre, name)
    u = 0.0 if name == "none" else ROUND[w.dtype]
    off = gz.abs() * u + 2.0 ** -20 * 1.2 * gy.to(F64).abs() + (STEP[w.dtype] if u else 0)
    size, (M, N) = gz.abs() + off, gz.shape
    sums = lambda s, k: 1.2 * (k / 16 + 32) * 2.0 ** -23 * s  # noqa: E731
    wx, ww, wb = gz @ w.to(F64), gz.t() @ x, gz.sum(0)
    _close(grads[0], wx, _out(wx, dtype, off @ w.to(F64).abs() + sums(size @ w.to(F64).abs(), N)), "grad_x")
    _close(grads[1], ww, _out(ww, dtype, off.t() @ x.abs() + sums(size.t() @ x.abs(), M)), "grad_w")
    own = (2.0 ** -20 * 1.2 * gy.to(F64).abs()).sum(0) if name != "none" else 0
    _close(grads[2], wb, own + (64 + M / 8) * E * gz.abs().sum(0), "grad_bias")


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu", "log1p_relu"])
@pytest.mark.parametrize("m,k,n", [(1, 64, 32), (3, 33, 5), (130, 640, 200), (257, 128, 256), (300, 1000, 1001), (1000, 104, 520)])
def test_linear_backward(h, dtype, name, m, k, n):
    x, w = _randn(m, k, dtype=dtype), _randn(n, k, std=k ** -0.5, dtype=dtype, seed=1)
    gy, pre = _randn(m, n, dtype=dtype, seed=2), _randn(m, n, std=2.0, dtype=dtype, seed=3)
    (qx, sx), (qp, sp) = h.compress(x), h.compress(pre)
    vx, vp = ref.stand_for(qx, sx), ref.stand_for(qp, sp)
    both = h.linear_backward(gy, qx, w, qp, name, x_scale=sx, pre_scale=sp)
    _check_layer(both, gy, vx, w, vp, name, dtype)
    again = h.linear_backward(gy, qx.contiguous(), w, qp.contiguous(), name, x_scale=sx, pre_scale=sp)
    assert all(torch.equal(a, b) for a, b in zip(both, again))
    if name != "none":
        _check_layer(h.linear_backward(gy, x, w, qp, name, pre_scale=sp, grad_dtype=torch.float32), gy, x.to(F64), w, vp, name, torch.float32)
    _check_layer(h.linear_backward(gy, qx, w, None if name == "none" else pre, name, x_scale=sx), gy, vx, w, pre.to(F64), name, dtype)


def test_linear_backward_by_differences(h):
    m, k, n, dtype = 40, 64, 72, torch.bfloat16
    x, w, gy = _randn(m, k, dtype=dtype), _randn(n, k, dtype=dtype, seed=1), _randn(m, n, dtype=dtype, seed=2)
    (qx, sx) = h.compress(x)
    vx = ref.stand_for(qx, sx).to(dtype)  # exact: a layer of these values
    _, qp, sp = h.linear(vx, w, activation="silu", compress_pre=True)
    gx, gw, _ = h.linear_backward(gy, qx, w, qp, "silu", x_scale=sx, pre_scale=sp, grad_dtype=torch.float32)
    f = {0: lambda v: dense.linear(v, w, None, "silu")[0], 1: lambda v: dense.linear(vx, v, None, "silu")[0]}
    for i, (at, grad) in enumerate(((vx, gx), (w, gw))):
        d, s = _randn(*at.shape, seed=5).to(F64), 2.0 ** -10
        up, down = ((gy.to(F64) * f[i](at.to(F64) + q * s * d)).sum() for q in (1, -1))
        # silu' changes by at most 1/2 of z's change, 2^-4 |z| (2^-10 of the
        # scale at most 2^-8 |z|_max below that); gz is then rounded to 8 bits
        z = dense.linear(vx, w)[1].abs()
        off = gy.to(F64).abs() * (0.5 * (2.0 ** -4 * z + 2.0 ** -17 * z.max()) + 1.1 * 2.0 ** -8)
        other = off @ w.to(F64).abs() if i == 0 else off.t() @ vx.to(F64).abs()
        assert abs(float(up - down) / (2 * s) - float((grad.to(F64) * d).sum())) <= float((other * d.abs()).sum())


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (2, 128), (5, 1001), (300, 96), (700, 1024), (4, 4096), (3, 8191), (2, 16384),
                                       (2, 20000), (1500, 520), (5000, 264)])
@pytest.mark.parametrize("more", [False, True])
def test_norm_backward(h, dtype, rows, cols, more):
    total, w = _randn(rows, cols, std=2.0, dtype=dtype), _randn(cols, seed=1)
    gy, gt = _randn(rows, cols, dtype=dtype, seed=2), _randn(rows, cols, dtype=dtype, seed=3) if more else None
    rstd = torch.rsqrt(total.float().square().mean(1) + 1e-6)
    q, s = h.compress(total)
    v = ref.stand_for(q, s)
    for weight in (w, w.to(dtype)):
        gx, gw = h.rms_norm_backward(gy, q, weight, rstd, gt, total_scale=s)
        wx, ww = dense.rms_norm_grad(gy, v, weight, rstd, gt)
        xh = v.abs() * rstd.to(F64)[:, None]
        g = gy.to(F64).abs() * weight.to(F64).abs()
        size = rstd.to(F64)[:, None] * (g + xh * (g * xh).mean(1, keepdim=True)) + (0 if gt is None else gt.to(F64).abs())
        _close(gx, wx, _out(wx, dtype, 64 * E * size), "grad_x")
        wsize = (gy.to(F64).abs() * xh).sum(0)
        _close(gw, ww, _out(ww, weight.dtype, (64 + rows / 8) * E * wsize), "grad_weight")
    again = h.rms_norm_backward(gy, q.contiguous(), w.to(dtype), rstd, gt, total_scale=s)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(40, 1032), (700, 2056), (9, 4104), (700, 5000), (5, 6152), (333, 7000), (700, 8192), (5, 8200)])
def test_norm_backward_of_wide_rows(h, dtype, rows, cols):
    test_norm_backward(h, dtype, rows, cols, True)


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_norm_backward_strides(h, pad, shift):
    for dtype in TYPES:
        total, w, gy = _randn(9, 520, dtype=dtype), _randn(520, seed=1), _randn(9, 520, dtype=dtype, seed=2)
        rstd = torch.rsqrt(total.float().square().mean(1) + 1e-6)
        q, s = h.compress(total)
        want = h.rms_norm_backward(gy, q, w, rstd, gy, total_scale=s)
        got = h.rms_norm_backward(_strided(gy, pad, shift), _strided(q, pad, shift), w, rstd, _strided(gy, pad), total_scale=s)
        v = ref.stand_for(q, s)
        wx, ww = dense.rms_norm_grad(gy, v, w, rstd, gy)
        size = wx.abs().max() * 4 + 4
        for gx, gw in (want, got):
            _close(gx, wx, _out(wx, dtype, 64 * E * size), "grad_x")
            _close(gw, ww, _out(ww, torch.float32, 72 * E * (gy.to(F64).abs() * v.abs() * rstd.to(F64)[:, None]).sum(0)), "grad_weight")


def test_norm_backward_no_rows(h):
    x = torch.empty(0, 64, device="cuda")
    q, s = h.compress(x)
    gx, gw = h.rms_norm_backward(x, q, torch.ones(64, device="cuda"), torch.empty(0, device="cuda"), total_scale=s)
    assert gx.shape == (0, 64) and not gw.any()


# ---------------------------------------------------------------- together
def test_a_training_step(h):
    """Norm, layer, cross entropy and back, everything kept in 8 bits, eagerly,
    on another stream and in a graph; with exact activations the gradients are
    near."""
    m, d, v, dtype = 200, 256, 3000, torch.bfloat16
    x, r = _randn(m, d, dtype=dtype), _randn(m, d, dtype=dtype, seed=1)
    g1, b1, w1 = 1 + 0.1 * _randn(d, seed=2), _randn(d, std=0.1, seed=3), _randn(d, d, std=d ** -0.5, dtype=dtype, seed=4)
    items, t = _randn(v, d, std=2.5 * d ** -0.5, dtype=dtype, seed=5), torch.randint(0, v, (m,), device="cuda")
    mean = torch.full((m,), 1.0 / m, device="cuda")

    def step(keep):
        y, total, rstd = h.rms_norm(x, g1, residual=r)
        if keep:
            a, pre, ps = h.linear(y, w1, bias=b1, activation="gelu", compress_pre=True)
            (y, ys), (total, ts) = h.compress(y), h.compress(total)
        else:
            a, pre = h.linear(y, w1, bias=b1, activation="gelu", save_pre=True)
            ps = ys = ts = None
        loss, ga, gv, _ = h.cross_entropy_step(a, items, t, mean)
        gy, gw, gb = h.linear_backward(ga, y, w1, pre, "gelu", x_scale=ys, pre_scale=ps)
        gx, gg = h.rms_norm_backward(gy, total, g1, rstd, total_scale=ts)
        return loss, gv, gw, gb, gx, gg

    plain, kept = step(False), step(True)
    assert torch.equal(plain[0], kept[0]) and torch.equal(plain[1], kept[1])
    for a, b in zip(plain[2:], kept[2:]):
        # each kept value is off by at most 2^-4 of itself, in either direction
        assert float((a.to(F64) - b.to(F64)).norm()) <= 2 * 2.0 ** -4 * float(a.to(F64).norm())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step(True)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(True)
    x.copy_(_randn(m, d, dtype=dtype, seed=9))
    fresh = step(True)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, fresh))


def test_refusals(h):
    from sparse_embedding_exact_gb300 import SparseCosError

    x, w, gy = _randn(20, 64, dtype=torch.bfloat16), _randn(40, 64, dtype=torch.bfloat16), _randn(20, 40, dtype=torch.bfloat16)
    q, s = h.compress(x)
    pre, ps = h.compress(gy)
    rstd, gain = torch.ones(20, device="cuda"), torch.ones(64, device="cuda")
    before = h.kernel_launches()
    bad = [(TypeError, lambda: h.expand(x, s)), (TypeError, lambda: h.expand(q, s.view(torch.uint8))),
           (ValueError, lambda: h.expand(q, s[:, :1])), (ValueError, lambda: h.expand(q, s[:5])), (TypeError, lambda: h.expand(q, None)),
           (ValueError, lambda: h.expand(q, s.cpu())), (ValueError, lambda: h.expand(q.t(), s)), (TypeError, lambda: h.expand(q, s, torch.int8)),
           (SparseCosError, lambda: h.compress(q)), (TypeError, lambda: h.compress(x.double())), (ValueError, lambda: h.compress(x[None])),
           (ValueError, lambda: h.linear(x, w, save_pre=True, compress_pre=True)),
           (SparseCosError, lambda: h.linear(x[:, :0], w[:, :0], compress_pre=True)),
           (SparseCosError, lambda: h.linear_backward(gy, x, w, None, "gelu", x_scale=None)),
           (TypeError, lambda: h.linear_backward(gy, x, w, pre, "gelu", x_scale=s, pre_scale=ps)),
           (TypeError, lambda: h.linear_backward(gy, q, w, None, "gelu", x_scale=s, pre_scale=ps)),
           (SparseCosError, lambda: h.linear_backward(gy, q, w, None, "gelu", x_scale=s)),
           (SparseCosError, lambda: h.linear_backward(gy.half(), q, w, pre, "gelu", x_scale=s, pre_scale=ps)),
           (SparseCosError, lambda: h.linear_backward(gy[:10], q, w, pre, "gelu", x_scale=s, pre_scale=ps)),
           (SparseCosError, lambda: h.linear_backward(gy, q[:, :32], w, pre, "gelu", x_scale=s[:, :1], pre_scale=ps)),
           (SparseCosError, lambda: h.rms_norm_backward(x[:10], q, gain, rstd, total_scale=s)),
           (TypeError, lambda: h.rms_norm_backward(x, x, gain, rstd, total_scale=s)),
           (SparseCosError, lambda: h.rms_norm_backward(x, q, gain, rstd, gy, total_scale=s))]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            print("not refused:", i)
    assert h.kernel_launches() == before
