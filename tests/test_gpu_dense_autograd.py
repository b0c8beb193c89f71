"""The dense operators beside torch's autograd: they are explicit calls outside
of it, and what is written in place says so."""
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


def _lists(rows, items, k):
    g = torch.Generator(device="cuda").manual_seed(0)
    return (torch.rand(rows, k, device="cuda", generator=g),
            torch.randint(0, items, (rows, k), device="cuda", generator=g))


def test_in_place_step_raises_the_version(h):
    z, lists = torch.randn(4, 100, device="cuda"), _lists(4, 100, 3)
    before = z._version
    h.distill_step(z, *lists)
    assert z._version == before  # only read
    _, grad = h.distill_step(z, *lists, in_place=True)
    assert grad is z and z._version > before


def test_overwritten_outputs_of_torch_are_noticed(h):
    # exp keeps its output for its gradient: the gradient in its place would
    # give other gradients, without torch's error
    a = torch.randn(4, 100, device="cuda", requires_grad=True)
    z = a.exp()
    _, grad = h.distill_step(z.detach(), *_lists(4, 100, 3), in_place=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward(grad)


def test_in_place_step_on_logits_with_a_gradient(h):
    # a product does not keep its output: the step in its place is a valid way
    lists = _lists(4, 100, 3)
    x, w = torch.randn(4, 8, device="cuda"), torch.randn(100, 8, device="cuda", requires_grad=True)
    _, want = h.distill_step((x @ w.detach().t()), *lists)
    z = x @ w.t()
    _, grad = h.distill_step(z, *lists, in_place=True)
    z.backward(grad.detach())
    assert torch.equal(grad.detach(), want)
    assert torch.allclose(w.grad, want.t() @ x, rtol=1e-5, atol=1e-6)


def test_in_place_step_in_inference_mode(h):
    lists = _lists(4, 100, 3)
    with torch.inference_mode():
        z = torch.randn(4, 100, device="cuda")
        _, want = h.distill_step(z, *lists)
        _, grad = h.distill_step(z, *lists, in_place=True)
    assert torch.equal(grad, want)
    _, grad = h.distill_step(z, *lists, in_place=True)  # outside of it too, as without a counter
    assert grad is z
