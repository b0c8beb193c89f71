"""GPU tests of the kept format where it is exact: codes and scales of a layer's
pre-activation bit for bit, whatever its sums and its neighbours are."""
import math

import pytest

torch = pytest.importorskip("torch")

import kept_reference as ref  # noqa: E402
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


def _randn(*shape, std=1.0, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def _small(*shape, seed=0):
    """Integers from -2 to 2."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, device="cuda", generator=g).float()


def _bias(n):
    """Groups whose largest value is 1.75 times a power of two, among borders
    between two codes and values beside them."""
    one = torch.tensor([448, 17, 19, 21, 23, -17, -19, 34, 38, -68, 1.0625, 1.1875, -1.3125, 272, 304, 0.0, 240, -248, 249,
                        17.03125, 18.96875, -33.9375, 2.0 ** -6, 2.0 ** -7 * 1.125, 2.0 ** -10, 2.0 ** -10 * 3, 5, 9, 11, 13, 15, -15],
                       device="cuda")
    groups = (n + 31) // 32
    return torch.cat([one * 2.0 ** (k % 5 - 3) for k in range(groups)])[:n].contiguous()


def _same(pre, scale, z, dtype):
    e = ref.exponents(z, ref.LEAST[dtype])
    q = ref.codes(z, e)
    got = pre.to(F64)
    assert torch.equal(ref.exponents_of(scale), e)
    assert torch.equal(torch.isnan(got), torch.isnan(q)) and torch.equal(got.nan_to_num(0.0), q.nan_to_num(0.0))


# Sums of integers far below 2^24 are exact in float32 in any order, and so are
# they with a bias of few bits: the codes are the 64-bit form's, ties included.
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,k,n", [(5, 64, 64), (70, 777, 200), (300, 1024, 1000), (40, 4096, 129), (600, 16_384, 320)])
def test_codes_of_exact_sums(h, dtype, m, k, n):
    x, w, b = _small(m, k).to(dtype), _small(n, k, seed=1).to(dtype), _bias(n)
    x[::3] = 0  # rows whose pre-activation is the bias
    z = x.to(F64) @ w.to(F64).t() + b.to(F64)
    assert torch.equal(z.float().to(F64), z) and float(z.abs().max()) < 2 ** 15
    y, pre, scale = h.linear(x, w, bias=b, activation="relu", out_dtype=dtype, compress_pre=True)
    _same(pre, scale, z, dtype)
    assert torch.equal(y, z.clamp_min(0).to(dtype))
    codes, again = h.compress(z.float())
    same = (ref.exponents(z, -126) == ref.exponents_of(scale)).repeat_interleave(32, 1)[:, :n]
    assert same.any() and torch.equal(codes.view(torch.uint8)[same], pre.view(torch.uint8)[same])


@pytest.mark.parametrize("dtype", HALVES)
def test_an_infinity_leaves_its_group(h, dtype):
    m, k, n = 70, 1024, 256
    x, w, b = _small(m, k).to(dtype), _small(n, k, seed=1).to(dtype), _bias(n)
    x[::3] = 0
    b[[5, 70, 100]] = math.inf
    b[[71, 200]] = -math.inf
    b[130] = math.nan
    z = x.to(F64) @ w.to(F64).t() + b.to(F64)
    _, pre, scale = h.linear(x, w, bias=b, activation="none", compress_pre=True)
    _same(pre, scale, z, dtype)


def test_codes_of_exact_sums_from_8_bits(h):
    m, k, n = 70, 512, 200
    x, w, b = _small(m, k).to(torch.float8_e4m3fn), _small(n, k, seed=1).to(torch.float8_e4m3fn), _bias(n)
    one = torch.ones(max(m, n), device="cuda")
    _, pre, scale = h.linear(x, w, bias=b, x_scale=one[:m], w_scale=0.5 * one[:n], compress_pre=True)
    _same(pre, scale, x.to(F64) @ w.to(F64).t() * 0.5 + b.to(F64), torch.bfloat16)


# Where the layer splits no sum (many tiles), the codes are those of the z that
# it keeps in float32, compressed in a call of its own: every one of them.
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("m,k,n", [(2100, 264, 2056), (2100, 777, 2056), (2304, 1024, 2304)])
def test_codes_as_compress_gives_them(h, dtype, m, k, n):
    x, w, b = _randn(m, k, dtype=dtype), _randn(n, k, std=k ** -0.5, dtype=dtype, seed=1), _randn(n, seed=2)
    _, pre, scale = h.linear(x, w, bias=b, activation="gelu", compress_pre=True)
    _, z = h.linear(x, w, bias=b, activation="gelu", out_dtype=torch.float32, save_pre=True)
    codes, want = h.compress(z)
    assert torch.equal(scale.view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(pre.view(torch.uint8), codes.view(torch.uint8))
