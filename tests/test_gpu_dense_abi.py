"""GPU tests of what only the C calls of the dense operators offer: the norm's
sum in one of its inputs' place, and gradients that are left out."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

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
        handle.check_device()


def _randn(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def _records(*tensors):
    from sparse_embedding_exact_gb300 import _abi

    code = {torch.float32: _abi.SS_VALUES_F32, torch.bfloat16: _abi.SS_VALUES_BF16, torch.float16: _abi.SS_VALUES_F16,
            torch.float8_e4m3fn: _abi.SS_VALUES_F8}
    out = []
    for t in tensors:
        rows, cols = (t.shape[0], t.shape[1]) if t.dim() == 2 else (1, t.shape[0])
        out.append(_abi.ss_dense(t.data_ptr(), rows, cols, t.stride(0) if rows > 1 else cols, code[t.dtype]))
    return out


def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(5, 7), (300, 256), (13_000, 1001), (50_000, 256), (400, 17_001)])
@pytest.mark.parametrize("place", ["x", "residual"])
@pytest.mark.parametrize("f8", [False, True])
def test_total_in_an_inputs_place(h, dtype, rows, cols, place, f8):
    x, r, w = _randn(rows, cols, dtype=dtype), _randn(rows, cols, dtype=dtype, seed=1), _randn(cols, dtype=dtype, seed=2)
    want_y, want_f, want_t = h.rms_norm_quantized(x, w, residual=r) if f8 else [h.rms_norm(x, w, residual=r)[i] for i in (0, 2, 1)]
    y, f = torch.empty_like(want_y), torch.empty_like(want_f)
    keep = _records(x, r, w, y)
    mx, mr, mw, my = (ctypes.addressof(m) for m in keep)
    mt = mx if place == "x" else mr
    scale, rstd = (f.data_ptr(), None) if f8 else (None, f.data_ptr())
    assert h._lib.ss_rms_norm(h._h, mx, mr, mw, 1e-6, mt, my, scale, rstd, _stream()) == 0
    total = x if place == "x" else r
    assert torch.equal(total, want_t) and torch.equal(f, want_f)
    assert torch.equal(y.view(torch.uint8), want_y.view(torch.uint8))


@pytest.mark.parametrize("m,k,n", [(3, 64, 40), (300, 1001, 77), (512, 256, 1024)])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("asked", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1), (0, 0, 0)])
def test_gradients_left_out(h, m, k, n, act, asked):
    from sparse_embedding_exact_gb300 import _abi
    from sparse_embedding_exact_gb300.dense import ACTIVATIONS

    dtype = torch.bfloat16
    x, w, gy = _randn(m, k, dtype=dtype), _randn(n, k, dtype=dtype, seed=1), _randn(m, n, dtype=dtype, seed=2)
    pre = _randn(m, n, dtype=dtype, seed=3)
    want = h.linear_backward(gy, x, w, pre if act != "none" else None, act)
    got = [torch.full_like(t, 7) for t in want]
    keep = _records(gy, x, w, pre, got[0], got[1])
    mg, mx, mw, mp, mgx, mgw = (ctypes.addressof(r) for r in keep)
    need = h._lib.ss_linear_backward_scratch(h._h, mg, mx, mw, ACTIVATIONS[act])
    room = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    st = h._lib.ss_linear_backward(h._h, mg, mx, mw, mp if act != "none" else None, ACTIVATIONS[act],
                                   mgx if asked[0] else None, mgw if asked[1] else None,
                                   got[2].data_ptr() if asked[2] else None, room.data_ptr(), need, _stream())
    assert st == _abi.SS_OK
    for a, g, wanted in zip(asked, got, want):
        assert torch.equal(g, wanted if a else torch.full_like(g, 7))
