"""The student of examples/distill_student.py learns the exact lists: the dense
operators together, as a program uses them."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_student_learns_the_teachers_lists():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_embedding_exact_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("distill_student", os.path.join(ROOT, "examples", "distill_student.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, before, after = example.train(steps=60, n_q=128, n_i=2000)
    # an untrained student is near the uniform distribution: log(2000) - entropy
    # of the teacher; half of it is far below
    assert losses[-1] < 0.5 * losses[0]
    assert after > before and after >= 0.5
