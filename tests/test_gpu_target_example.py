"""The example of a student trained on chosen items runs, and its gradients are
those of its loss, as torch finds them for a 64-bit form: with 16-bit
activations within the roundings on the way, with 8-bit ones within theirs."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_embedding_exact_gb300 import build

    build.build()


def test_runs(ready):
    from examples import target_student

    losses = target_student.train(steps=3, n_q=64, n_i=500)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)


def test_gradients(ready):
    import sparse_embedding_exact_gb300 as sec
    from examples import target_student as ex

    d, dev = torch.float64, torch.device("cuda", 0)
    with sec.SparseCosine(ex.CONFIGS["d65k_q1k_i10k"].dim) as h:
        x, chosen, popularity = ex.chosen_items(h, 48, 300, dev)
        p, mean = ex.start(300, dev), torch.full((48,), 1.0 / 48, device=dev)
        losses, grads = ex.forward_backward(h, p, x, chosen, popularity, mean, keep=False)
        kept_losses, kept = ex.forward_backward(h, p, x, chosen, popularity, mean, keep=True)
        assert torch.equal(losses, kept_losses)  # the forward pass is the same

        leaves = {k: v.to(ex.BF16).to(d).requires_grad_() if k in ("w1", "v") else v.to(d).requires_grad_() for k, v in p.items()}

        def norm(t, g):
            return t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6) * g

        y = norm(x.to(d), leaves["g1"])
        a = torch.nn.functional.gelu(y @ leaves["w1"].t() + leaves["b1"])
        z = norm(a + x.to(d), leaves["g2"]) @ leaves["v"].t() + popularity.to(d)
        want_loss = torch.nn.functional.cross_entropy(z, chosen, reduction="none")
        want = torch.autograd.grad((want_loss * mean.to(d)).sum(), list(leaves.values()))
        # five roundings to 8 bits on the way (y, a, the sum, y2, its gradient
        # and gz) reach a logit of size up to 10 and then each gradient: 2^-8 of
        # it each, here summed as if they all went one way
        assert float((losses.to(d) - want_loss.detach()).abs().max()) <= 5 * 2.0 ** -8 * float(z.detach().abs().max())
        for (name, got), w in zip(grads.items(), want):
            far = float((got.to(d) - w).norm() / w.norm())
            assert far <= 10 * 2.0 ** -8, (name, far)
            # kept in 8 bits: 2^-4 of an activation, of which the norm's gradient
            # and the slope see two and the layer's weights one, on the way back
            kept_far = float((kept[name].to(d) - w).norm() / w.norm())
            assert kept_far <= 10 * 2.0 ** -8 + 4 * 2.0 ** -4, (name, kept_far)
