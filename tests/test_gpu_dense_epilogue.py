"""GPU tests of what a linear layer does after its product, where everything is
exact: integers in, so that each output is the 64-bit form's, rounded once."""
import pytest

torch = pytest.importorskip("torch")

from dense_reference import F64  # noqa: E402

pytestmark = pytest.mark.gpu
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


def _ints(low, high, *shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(low, high, shape, device="cuda", generator=g).float()


def _strided(t, pad, shift):
    """t as part of a larger matrix of another value everywhere."""
    buf = torch.full((t.shape[0] * (t.shape[1] + pad) + shift + 16,), 77.0, device=t.device).to(t.dtype)
    v = buf.as_strided(t.shape, (t.shape[1] + pad, 1), shift)
    v.copy_(t)
    return v


# Rows and features at the edges of boxes of 32 x 32, of tiles and of many tiles a
# pair of blocks.
SHAPES = [(300, 64, 200), (257, 72, 520), (1000, 40, 1001), (2100, 64, 2056), (2305, 24, 2049), (6000, 64, 2080), (130, 512, 96), (33, 64, 64)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,k,n", SHAPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 1)])
def test_residual_and_pre_activation(h, dtype, m, k, n, pad, shift):
    x, w, b = _ints(-2, 3, m, k).to(dtype), _ints(-2, 3, n, k, seed=1).to(dtype), _ints(-8, 9, n, seed=2) / 4
    r = _ints(-100, 101, m, n, seed=3)
    z = x.to(F64) @ w.to(F64).t() + b.to(F64)
    relu = z.clamp_min(0)
    for out in (dtype, torch.float32):
        res = _strided(r.to(out), pad, shift)
        for act, a in (("none", z), ("relu", relu)):
            want = (a + r.to(F64)).float().to(out)
            for keep in (False, True):
                got = h.linear(x, w, bias=b, activation=act, residual=res, out_dtype=out, save_pre=keep)
                y = got[0] if keep else got
                assert torch.equal(y, want)
                if keep:
                    assert torch.equal(got[1], z.float().to(out))
            y, pre = h.linear(x, w, bias=b, activation=act, out_dtype=out, save_pre=True)
            assert torch.equal(y, a.float().to(out)) and torch.equal(pre, z.float().to(out))
            y, _, _ = h.linear(x, w, bias=b, activation=act, residual=res, out_dtype=out, compress_pre=True)
            assert torch.equal(y, want)
            assert torch.equal(h.linear(x, w, bias=b, activation=act, out_dtype=out), a.float().to(out))


def test_residual_changes_with_every_call(h):
    """Boxes fetched ahead belong to their own tile: another residual, other values."""
    m, k, n, dtype = 5000, 64, 4096, torch.bfloat16
    x, w = _ints(-2, 3, m, k).to(dtype), _ints(-2, 3, n, k, seed=1).to(dtype)
    z = x.to(F64) @ w.to(F64).t()
    side = torch.cuda.Stream()
    for seed in range(4):
        r = _ints(-100, 101, m, n, seed=seed).to(dtype)
        want = (z + r.to(F64)).float().to(dtype)
        assert torch.equal(h.linear(x, w, residual=r), want)
        side.wait_stream(torch.cuda.current_stream())
        y, pre = h.linear(x, w, residual=r, save_pre=True, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, want) and torch.equal(pre, z.float().to(dtype))


# Few rows and many features, whose sums go by shares; one and many slices of
# 256 columns; odd widths.
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,k,n", [(1, 1024, 4096), (16, 4096, 4096), (70, 1000, 3000), (200, 257, 10_000), (65, 777, 2049), (600, 512, 1000)])
def test_gradients_of_exact_sums(h, dtype, m, k, n):
    x, w, gy = _ints(-2, 3, m, k).to(dtype), _ints(-2, 3, n, k, seed=1).to(dtype), _ints(-2, 3, m, n, seed=2).to(dtype)
    pre = _ints(-1, 2, m, n, seed=3).to(dtype)
    for act, gz in (("none", gy.to(F64)), ("relu", gy.to(F64) * (pre > 0))):
        gx, gw, gb = h.linear_backward(gy, x, w, None if act == "none" else pre, act, grad_dtype=torch.float32)
        assert torch.equal(gx.to(F64), gz @ w.to(F64)) and torch.equal(gw.to(F64), gz.t() @ x.to(F64)) and torch.equal(gb.to(F64), gz.sum(0))
        gx, gw, _ = h.linear_backward(gy, x, w, None if act == "none" else pre, act)
        assert torch.equal(gx, (gz @ w.to(F64)).float().to(dtype)) and torch.equal(gw, (gz.t() @ x.to(F64)).float().to(dtype))
