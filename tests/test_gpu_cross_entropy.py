"""GPU tests of the cross entropy over every item against its 64-bit form, with
the bounds that xent_reference derives."""
import math

import pytest

torch = pytest.importorskip("torch")

import xent_reference as ref  # noqa: E402
from dense_reference import F64  # noqa: E402

pytestmark = pytest.mark.gpu
HALVES = [torch.bfloat16, torch.float16]
NAMES = ("loss", "grad_x", "grad_w", "grad_bias")


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
    if "h" in request.fixturenames and request.node.name != "test_target_past_the_end":
        request.getfixturevalue("h").check_device()


def _randn(*shape, std=1.0, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def _strided(t, pad, shift=0):
    buf = torch.full((t.shape[0] * (t.shape[1] + pad) + shift + 16,), float("nan"), device=t.device).to(t.dtype)
    v = buf.as_strided(t.shape, (t.shape[1] + pad, 1), shift)
    v.copy_(t)
    return v


def _case(m, v, k, dtype, seed=0, std=2.5):
    x, w = _randn(m, k, dtype=dtype, seed=seed), _randn(v, k, std=std * k ** -0.5, dtype=dtype, seed=seed + 1)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    t = torch.randint(0, v, (m,), device="cuda", generator=g)
    return x, w, t, _randn(v, std=0.5, seed=seed + 3), torch.rand(m, device="cuda", generator=g) + 0.5, _randn(m, seed=seed + 4)


def _compare(got, want, room, what=""):
    got = got.to(F64)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - room
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: over the bound by {float(over.max())}"


def _check(h, x, w, t, gl, bias=None, weight=None, T=1.0, dtype=None, plain=None, pieces=1, given=None):
    """Forward, backward and step against the 64-bit form of `plain` (x, w where
    these are strided)."""
    px, pw = plain or (x, w)
    more = dict(bias=bias, weight=weight, temperature=T)
    r = ref.cross_entropy(px, pw, t, gl, **more)
    room = ref.bounds(r, px, pw, bias, weight, gl, T, dtype, pieces)
    loss, stats = h.cross_entropy(x, w, t, **more)
    gx, gw, gb = h.cross_entropy_backward(gl, x, w, t, stats, grad_dtype=dtype, **more)
    step = h.cross_entropy_step(x, w, t, gl, grad_dtype=dtype, **more)
    for name, a, b in zip(NAMES, (loss, gx, gw, gb), step):
        if a is None:
            assert b is None and bias is None and name == "grad_bias"
            continue
        _compare(a, r[name], room[name], name)
        assert torch.equal(a, b), f"{name}: step differs"
    assert gx.dtype == gw.dtype == (dtype or x.dtype) and loss.dtype == torch.float32
    return r, (loss, stats, gx, gw, gb)


SHAPES = [(1, 1, 1), (1, 1000, 64), (2, 7, 3), (3, 255, 8), (5, 256, 63), (31, 257, 64), (33, 1000, 65), (128, 300, 200),
          (129, 513, 72), (256, 512, 128), (257, 2049, 136), (300, 5000, 24), (700, 10_000, 256), (16, 30_000, 104)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,v,k", SHAPES)
def test_cross_entropy(h, dtype, m, v, k):
    x, w, t, b, wt, gl = _case(m, v, k, dtype)
    _check(h, x, w, t, gl, b, wt)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T", [0.05, 0.5, 4.0])
@pytest.mark.parametrize("out", [None, torch.float32])
def test_temperatures_and_types(h, dtype, T, out):
    x, w, t, b, wt, gl = _case(150, 700, 96, dtype, std=2.5 * min(T, 1.0))
    _check(h, x, w, t, gl, b * T, wt, T, out)
    _check(h, x, w, t, None, None, None, T, out)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_strides(h, dtype, pad, shift):
    x, w, t, b, wt, gl = _case(70, 400, 72, dtype)
    _check(h, _strided(x, pad, shift), _strided(w, 2 * pad, shift), t, gl, b, wt, plain=(x, w))


@pytest.mark.parametrize("which", ["x", "w"])
def test_one_of_two_needs_a_copy(h, which):
    # one matrix's rows start on 16-byte boundaries, the other's do not
    for dtype in HALVES:
        x, w, t, b, wt, gl = _case(70, 400, 72, dtype)
        xs, ws = (_strided(x, 3), w) if which == "x" else (x, _strided(w, 3))
        _check(h, xs, ws, t, gl, b, wt, plain=(x, w))


def test_absent_rows_and_masked_items(h):
    for dtype in HALVES:
        x, w, t, b, wt, gl = _case(300, 600, 64, dtype)
        b[::7] = -math.inf
        b[t[20:]] = 0.25
        t[3], wt[9], t[11] = -1, 0.0, -5
        b[50] = -math.inf
        t[13] = 50  # its target is masked
        r = ref.cross_entropy(x, w, t, gl, b, wt)
        dead = torch.tensor([3, 9, 11, 13], device="cuda")
        assert not r["live"][dead].any() and int(r["live"].sum()) > 200
        x2 = x.clone()
        x2[[3, 11]] = math.nan
        x2[9] = math.inf
        _, (loss, stats, gx, gw, gb) = _check(h, x2, w, t, gl, b, wt, plain=(x, w))
        assert not loss[dead].any() and not gx[dead].any()
        masked = torch.isinf(b)
        assert not gw[masked].any() and not gb[masked].any()


def test_rows_of_masked_targets_hold_anything(h):
    for dtype in HALVES:
        x, w, t, b, wt, gl = _case(70, 600, 64, dtype)
        b[77] = -math.inf
        t[[4, 40, 69]] = 77
        b[t[:3]] = 0.0
        clean = x.clone()
        clean[[4, 40, 69]] = 0.0
        x[4], x[40, 5], x[69] = math.nan, math.inf, -math.inf
        _, (loss, _, gx, _, _) = _check(h, x, w, t, gl, b, wt, plain=(clean, w))
        assert not loss[[4, 40, 69]].any() and not gx[[4, 40, 69]].any()


def test_padded_rows_have_any_weight_and_gradient(h):
    # rows that take no part do not set the scale of those that do
    for dtype in HALVES:
        x, w, t, b, wt, gl = _case(70, 600, 64, dtype)
        b[77] = -math.inf
        t[[4, 40]] = -1
        t[[5, 69]] = 77
        wt[50] = 0.0
        b[t[:3]] = 0.0
        plain = [v.clone() for v in (wt, gl)]
        r = ref.cross_entropy(x, w, t, plain[1], b, plain[0])
        room = ref.bounds(r, x, w, b, plain[0], plain[1])
        wt[[4, 5]], gl[[4, 69]], gl[50] = 1e30, 1e25, 1e35
        wt[40], gl[40] = math.nan, math.inf
        got = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt)
        for name, one in zip(NAMES, got):
            _compare(one, r[name], room[name], name)
        _, stats = h.cross_entropy(x, w, t, bias=b, weight=wt)
        for name, one in zip(NAMES[1:], h.cross_entropy_backward(gl, x, w, t, stats, bias=b, weight=wt)):
            _compare(one, r[name], room[name], name)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,mask", [(1.0, torch.finfo(torch.float32).min), (4.0, torch.finfo(torch.bfloat16).min), (0.05, -5e36), (0.05, -3e38)])
def test_masks_of_the_lowest_value(h, dtype, T, mask):
    # whole units, tiles and halves of tiles of masked items, and a row's target among them
    x, w, t, b, wt, gl = _case(300, 3000, 64, dtype)
    b[300:1700], b[1800:1835], b[2990:] = -math.inf, -math.inf, -math.inf
    t[:] = t % 250
    t[7], t[200] = 301, 2995
    low = torch.where(torch.isinf(b), torch.full_like(b, mask), b)
    b[::5], low[::5] = -math.inf, -math.inf
    _, want = _check(h, x, w, t, gl, b, wt, T=T)
    loss, stats = h.cross_entropy(x, w, t, bias=low, weight=wt, temperature=T)
    got = (loss, stats) + tuple(h.cross_entropy_backward(gl, x, w, t, stats, bias=low, weight=wt, temperature=T))
    assert not loss[[7, 200]].any() and loss.count_nonzero() > 200
    for a, one in zip(want, got):
        assert torch.equal(a, one)
    for a, one in zip((want[0],) + tuple(want[2:]), h.cross_entropy_step(x, w, t, gl, bias=low, weight=wt, temperature=T)):
        assert torch.equal(a, one)
    everything = torch.full_like(b, mask)
    assert not any(o.any() for o in h.cross_entropy_step(x, w, t, gl, bias=everything, weight=wt, temperature=T))


def test_everything_masked(h):
    x, w, t, b, wt, gl = _case(40, 300, 32, torch.bfloat16)
    loss, stats = h.cross_entropy(x, w, t, bias=torch.full_like(b, -math.inf))
    assert not loss.any()
    out = h.cross_entropy_step(x, w, t, gl, bias=torch.full_like(b, -math.inf), weight=wt)
    assert not any(o.any() for o in out)
    t[:] = -1
    assert not any(o.any() for o in h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt))


def test_target_past_the_end(h):
    from sparse_embedding_exact_gb300 import SparseCosError

    x, w, t, b, wt, gl = _case(40, 300, 32, torch.bfloat16)
    t[5], t[6] = 300, 2 ** 40
    r = ref.cross_entropy(x, w, t, gl, b, wt)
    room = ref.bounds(r, x, w, b, wt, gl)
    for name, got in zip(NAMES, h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt)):
        _compare(got, r[name], room[name], name)
    assert not r["live"][[5, 6]].any()
    with pytest.raises(SparseCosError):
        h.check_device()
    h.check_device()


def test_far_logits(h):
    # a softmax that is nearly one item, and items whose softmax is 0
    x, w, t, b, wt, gl = _case(100, 500, 64, torch.bfloat16, std=60.0)
    _check(h, x, w, t, gl, b, wt)


def test_small_gradients_in_float16(h):
    # the gradient of a mean over many rows: most of gz lies below binary16's
    # smallest values, and some rows' far below the others'
    x, w, t, b, wt, gl = _case(200, 3000, 64, torch.float16)
    for size in (1e-7, 1e-4, 1e5):
        _check(h, x, w, t, gl * size, b, wt, dtype=torch.float32)
    assert not any(o.any() for o in h.cross_entropy_step(x, w, t, gl * 0, bias=b, weight=wt)[1:])


def test_special_values(h):
    x, w, t, b, wt, gl = _case(40, 300, 32, torch.bfloat16)
    x[7, 3] = math.nan
    loss, gx, gw, gb = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt)
    assert torch.isnan(loss).nonzero().flatten().tolist() == [7]
    assert torch.isnan(gx).all(1).nonzero().flatten().tolist() == [7] and not torch.isnan(gx[:7]).any()
    assert torch.isnan(gb).all() and torch.isnan(gw).all()


# More values of gz than one piece holds, and many tiles a pair of blocks
@pytest.mark.parametrize("dtype,m,v,k,out", [(torch.bfloat16, 4200, 65_000, 64, None), (torch.float16, 2100, 70_001, 40, torch.float32),
                                             (torch.bfloat16, 9000, 20_003, 136, None)])
def test_pieces(h, dtype, m, v, k, out):
    x, w, t, b, wt, gl = _case(m, v, k, dtype)
    _check(h, x, w, t, gl, b, wt, dtype=out, pieces=1 + m * v // 2 ** 27)


def test_gradient_by_differences(h):
    m, v, k = 40, 90, 24
    x, w, t, b, wt, gl = _case(m, v, k, torch.bfloat16)
    _, gx, gw, gb = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt, temperature=0.7, grad_dtype=torch.float32)
    f = {0: lambda a: ref.cross_entropy(a, w, t, gl, b, wt, 0.7)["loss"], 1: lambda a: ref.cross_entropy(x, a, t, gl, b, wt, 0.7)["loss"],
         2: lambda a: ref.cross_entropy(x, w, t, gl, a, wt, 0.7)["loss"]}
    for i, (at, grad) in enumerate(((x, gx), (w, gw), (b, gb))):
        d, s = _randn(*at.shape, seed=5).to(F64), 2.0 ** -12
        up, down = ((gl.to(F64) * f[i](at.to(F64) + q * s * d)).sum() for q in (1, -1))
        # gz is rounded to 8 bits: 2^-8 of each of its products with d's values
        r = ref.cross_entropy(x, w, t, gl, b, wt, 0.7)
        other = {0: r["gz"].abs() @ w.to(F64).abs(), 1: r["gz"].abs().t() @ x.to(F64).abs(), 2: r["gz"].abs().sum(0)}[i]
        assert abs(float(up - down) / (2 * s) - float((grad.to(F64) * d).sum())) <= 2.0 ** -8 * float((other * d.abs()).sum())


def test_no_rows(h):
    x, w = torch.empty(0, 24, device="cuda", dtype=torch.bfloat16), _randn(50, 24, dtype=torch.bfloat16)
    t, b = torch.empty(0, dtype=torch.int64, device="cuda"), _randn(50)
    loss, gx, gw, gb = h.cross_entropy_step(x, w, t, bias=b)
    assert loss.shape == (0,) and gx.shape == (0, 24) and gw.shape == (50, 24) and not gw.any() and not gb.any()
    assert h.cross_entropy(x, w, t)[1].shape == (0, 2)


def test_streams_and_graphs(h):
    x, w, t, b, wt, gl = _case(300, 3000, 128, torch.float16)
    want = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt)
    x2, w2, t2, b2, wt2, gl2 = _case(300, 3000, 128, torch.float16, seed=50)
    fresh = h.cross_entropy_step(x2, w2, t2, gl2, bias=b2, weight=wt2)
    for old, new in ((x, x2), (w, w2), (t, t2), (b, b2), (wt, wt2), (gl, gl2)):
        old.copy_(new)
    for _ in range(2):
        for o in out:
            o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, fresh))


def test_two_streams_at_once(h):
    cases = [_case(500, 6000, 200, dtype, seed=10 * i) for i, dtype in enumerate(HALVES)]
    want = [h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt) for x, w, t, b, wt, gl in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for s, (x, w, t, b, wt, gl) in zip(streams, cases):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt) for _ in range(8)])
    torch.cuda.synchronize()
    for outs, one in zip(got, want):
        for out in outs:
            assert all(torch.equal(p, q) for p, q in zip(out, one))


def test_calls_in_a_row_share_memory(h):
    # each call's scratch is the one before's, freed and taken again: no kernel
    # of a call starts on it early
    cases = [_case(m, v, k, torch.bfloat16, seed=m) for m, v, k in ((600, 9000, 96), (40, 20_000, 72), (1500, 3000, 260))]
    want = [h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt) for x, w, t, b, wt, gl in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for (x, w, t, b, wt, gl), one in zip(cases, want):
            out = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt)
            assert all(torch.equal(p, q) for p, q in zip(out, one))


@pytest.mark.parametrize("v", [2561, 2592, 2593, 2624, 2625])
def test_last_columns_over_many_tiles(h, v):
    # tiles whose last quarter, or half of one, has no columns, many a pair of blocks
    x, w, t, b, wt, gl = _case(5000, v, 64, torch.bfloat16)
    _, (_, _, gx, gw, gb) = _check(h, x, w, t, gl, b, wt)
    for _ in range(5):
        again = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt)
        assert all(torch.equal(p, q) for p, q in zip(again[1:], (gx, gw, gb)))


def test_gradients_left_out(h):
    # the C calls' NULL gradients: the others' bits stay, and what is left out is not written
    import ctypes

    from sparse_embedding_exact_gb300 import _abi

    x, w, t, b, wt, gl = _case(300, 2000, 136, torch.float16)
    want = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt)

    def record(m):
        return _abi.ss_dense(m.data_ptr(), m.shape[0], m.shape[1], m.stride(0), _abi.SS_VALUES_F16)

    for asked in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1), (0, 0, 0)):
        got = [torch.full_like(g, 7) for g in want]
        keep = [record(m) for m in (x, w, got[1], got[2])]
        at = [ctypes.addressof(r) for r in keep]
        need = h._lib.ss_cross_entropy_step_scratch(h._h, at[0], at[1])
        room = torch.empty(need, dtype=torch.uint8, device="cuda")
        st = h._lib.ss_cross_entropy_step(h._h, gl.data_ptr(), at[0], at[1], b.data_ptr(), t.data_ptr(), 1.0, wt.data_ptr(),
                                          got[0].data_ptr(), at[2] if asked[0] else None, at[3] if asked[1] else None,
                                          got[3].data_ptr() if asked[2] else None, room.data_ptr(), need,
                                          torch.cuda.current_stream().cuda_stream)
        assert st == _abi.SS_OK
        assert torch.equal(got[0], want[0])
        for a, g, one in zip(asked, got[1:], want[1:]):
            assert torch.equal(g, one if a else torch.full_like(g, 7))
        st = h._lib.ss_cross_entropy_step(h._h, gl.data_ptr(), at[0], at[1], b.data_ptr(), t.data_ptr(), 1.0, wt.data_ptr(),
                                          got[0].data_ptr(), at[2], at[3], got[3].data_ptr(), room.data_ptr(), need - 1,
                                          torch.cuda.current_stream().cuda_stream)
        assert st == _abi.SS_ERR_INVALID_ARG


def test_refusals(h):
    from sparse_embedding_exact_gb300 import SparseCosError

    x, w, t, b, wt, gl = _case(40, 300, 32, torch.bfloat16)
    loss, stats = h.cross_entropy(x, w, t)
    before = h.kernel_launches()
    bad = [(SparseCosError, lambda: h.cross_entropy(x.float(), w.float(), t)), (SparseCosError, lambda: h.cross_entropy(x, w.half(), t)),
           (SparseCosError, lambda: h.cross_entropy(x, w[:, :16], t)), (SparseCosError, lambda: h.cross_entropy(x, w[:0], t)),
           (SparseCosError, lambda: h.cross_entropy(x[:, :0], w[:, :0], t)),
           (SparseCosError, lambda: h.cross_entropy(x, w, t, temperature=0.0)),
           (SparseCosError, lambda: h.cross_entropy(x, w, t, temperature=math.nan)),
           (TypeError, lambda: h.cross_entropy(x, w, t.int())), (ValueError, lambda: h.cross_entropy(x, w, t[:3])),
           (TypeError, lambda: h.cross_entropy(x, w, None)), (ValueError, lambda: h.cross_entropy(x, w, t.cpu())),
           (ValueError, lambda: h.cross_entropy(x, w, t, bias=b[:-1])), (TypeError, lambda: h.cross_entropy(x, w, t, bias=b.half())),
           (ValueError, lambda: h.cross_entropy(x, w, t, weight=wt[1:])), (ValueError, lambda: h.cross_entropy(x.t(), w, t)),
           (TypeError, lambda: h.cross_entropy_backward(gl, x, w, t, None)),
           (ValueError, lambda: h.cross_entropy_backward(gl, x, w, t, stats[:4])),
           (ValueError, lambda: h.cross_entropy_step(x, w, t, gl[:4])),
           (TypeError, lambda: h.cross_entropy_step(x, w, t, gl, grad_dtype=torch.float64)),
           (SparseCosError, lambda: h.cross_entropy_step(x, w, t, gl, grad_dtype=torch.float16))]
    for error, call in bad:
        with pytest.raises(error):
            call()
    assert h.kernel_launches() == before
