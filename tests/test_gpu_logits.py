"""GPU tests of the cross entropy's logits: wide sums, exact ones among them, and
values that are not numbers."""
import math

import pytest

torch = pytest.importorskip("torch")

import xent_reference as ref  # noqa: E402
from dense_reference import F64  # noqa: E402

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
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
        handle.check_device()


def _randn(*shape, std=1.0, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def _ints(low, high, *shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(low, high, shape, device="cuda", generator=g)


# Logits that float32 holds exactly in any order of their sums: rows of x with
# one or a few ones, and of small integers.  No sum is off then, so a row's
# largest logit is exact, and the loss is off by its exponentials and their sum
# alone, as `bounds` counts them.
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,v,k", [(70, 500, 64), (70, 500, 777), (300, 500, 2048), (40, 300, 16_384)])
@pytest.mark.parametrize("masked", [False, True])
def test_exact_logits(h, dtype, m, v, k, masked):
    x = torch.zeros(m, k, device="cuda", dtype=dtype)
    x.scatter_(1, _ints(0, k, m, 1), 1)
    x[::3] = 0
    x[::3].scatter_(1, _ints(0, k, len(x[::3]), 3, seed=1), 1)
    x[::5] = _ints(-1, 2, len(x[::5]), k, seed=2).to(dtype) * (_ints(0, k, len(x[::5]), k, seed=3) < 8).to(dtype)
    w, t = _ints(-12, 13, v, k, seed=4).to(dtype), _ints(0, v, m, seed=5)
    b = _ints(-8, 9, v, seed=6).float() / 8
    if masked:
        b[::3] = -math.inf
        t = t // 3 * 3 + 1
        t = torch.where(t < v, t, torch.ones_like(t))
    z = x.to(F64) @ w.to(F64).t() + b.to(F64)
    loss, stats = h.cross_entropy(x, w, t, bias=b)
    assert torch.equal(stats[:, 0].to(F64), z.amax(1))
    r = ref.cross_entropy(x, w, t, None, b)
    reach = (z.amax(1) - z.masked_fill(torch.isinf(z), math.inf).amin(1)) * 1.45
    room = 3 * E * reach + (v / 7 + 64) * E + 8 * E * (1 + reach + r["loss"].abs())
    assert ((loss.to(F64) - r["loss"]).abs() <= room).all()
    total = torch.exp(z - z.amax(1, keepdim=True)).sum(1)
    assert ((stats[:, 1].to(F64) - total).abs() <= (3 * E * reach + (v / 7 + 64) * E) * total).all()


# The logits are the sums that the layer's calls give: where these split no sum
# (many tiles), a row's largest is the same bits.
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("k", [264, 777, 1024, 2048])
def test_logits_are_the_layers(h, dtype, k):
    m, v = 2304, 2304
    x, w, b = _randn(m, k, dtype=dtype), _randn(v, k, std=2.5 * k ** -0.5, dtype=dtype, seed=1), _randn(v, std=0.5, seed=2)
    _, stats = h.cross_entropy(x, w, _ints(0, v, m), bias=b)
    z = h.linear(x, w, bias=b, out_dtype=torch.float32)
    assert torch.equal(stats[:, 0], z.amax(1))


def _compare(got, want, room, what):
    got = got.to(F64)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - room
    assert float(over.max()) <= 0, f"{what}: over the bound by {float(over.max())}"


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,v,k,T", [(130, 700, 777, 0.5), (300, 1000, 1024, 1.0), (70, 600, 2048, 2.0), (40, 300, 16_400, 1.0)])
def test_wide_sums(h, dtype, m, v, k, T):
    x, w = _randn(m, k, dtype=dtype), _randn(v, k, std=2.5 * T * k ** -0.5, dtype=dtype, seed=1)
    b, t, wt, gl = _randn(v, std=0.5, seed=2), _ints(0, v, m, seed=3), _randn(m, seed=4).abs() + 0.5, _randn(m, seed=5)
    r = ref.cross_entropy(x, w, t, gl, b, wt, T)
    room = ref.bounds(r, x, w, b, wt, gl, T)
    got = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt, temperature=T)
    for name, one in zip(NAMES, got):
        _compare(one, r[name], room[name], name)


# Items whose logits are not numbers, alone or among masked ones: where a thread's
# first 32 columns, a block's or a unit's have no other, and in a last, short block.
NOT_NUMBERS = [(1000, range(0, 32)), (1000, range(32, 64)), (1000, range(0, 64)), (1000, range(256, 512)), (3000, range(0, 2816)),
               (33, [32]), (257, [256]), (1, [0]), (700, [699]), (700, [300])]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("m", [1, 300])
@pytest.mark.parametrize("v,items", NOT_NUMBERS)
def test_a_nan_shows(h, m, v, items, masked):
    for dtype in HALVES:
        x, w, t = _randn(m, 64, dtype=dtype), _randn(v, 64, std=0.3, dtype=dtype, seed=1), _ints(0, v, m, seed=2)
        b, wt = torch.zeros(v, device="cuda"), torch.ones(m, device="cuda")
        items = list(items)
        if masked and len(items) > 1:  # all but one of them
            b[items[1:]] = -math.inf
        w[items[:1] if masked else items] = math.nan
        live = torch.ones(m, dtype=torch.bool, device="cuda")
        if m > 8:
            t[3], wt[5] = -1, 0.0
            live[[3, 5]] = False
        live &= ~torch.isinf(b[t.clamp_min(0)])
        loss, stats = h.cross_entropy(x, w, t, bias=b, weight=wt)
        step = h.cross_entropy_step(x, w, t, bias=b, weight=wt)
        assert torch.equal(torch.isnan(loss), live) and not loss[~live].any()
        assert torch.equal(torch.isnan(step[0]), live) and not step[0][~live].any()
        for gx in (step[1], h.cross_entropy_backward(None, x, w, t, stats, bias=b, weight=wt)[0]):
            assert torch.isnan(gx[live]).all()


def test_rows_past_a_piece(h):
    """More rows than 2^27 values of the least piece of items have."""
    m, v, k, dtype = 70_000, 4500, 40, torch.bfloat16
    x, w = _randn(m, k, dtype=dtype), _randn(v, k, std=2.5 * k ** -0.5, dtype=dtype, seed=1)
    b, t, wt, gl = _randn(v, std=0.5, seed=2), _ints(0, v, m, seed=3), _randn(m, seed=4).abs() + 0.5, _randn(m, seed=5)
    t[::1000], wt[7::900] = -1, 0.0
    r = ref.cross_entropy(x, w, t, gl, b, wt)
    room = ref.bounds(r, x, w, b, wt, gl, pieces=3)
    got = h.cross_entropy_step(x, w, t, gl, bias=b, weight=wt)
    for name, one in zip(NAMES, got):
        _compare(one, r[name], room[name], name)
