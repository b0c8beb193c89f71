"""The dense operators' scratch queries on the host: they need no GPU, only a
handle's SM count.  Run in a process of its own, which a fault of the query
would end."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import ctypes, sys
from sparse_embedding_exact_gb300 import _abi
lib = _abi.load()
handle = (ctypes.c_char * (1 << 20))()  # a handle of zeros: no SM known
m, n, k = (int(v) for v in sys.argv[1:4])

def matrix(rows, cols):
    return _abi.ss_dense(None, rows, cols, cols, _abi.SS_VALUES_BF16)

gy, x, w = matrix(m, n), matrix(m, k), matrix(n, k)
at = ctypes.addressof
for act in (_abi.SS_ACT_NONE, _abi.SS_ACT_GELU):
    print(lib.ss_linear_backward_scratch(at(handle), at(gy), at(x), at(w), act))
print(lib.ss_linear_scratch(at(handle), at(x), at(w)))
print(lib.ss_rms_norm_backward_scratch(at(handle), m, k))
"""


def _scratch(m, n, k):
    from sparse_embedding_exact_gb300 import build

    build.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(m), str(n), str(k)], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr)
    return [int(v) for v in r.stdout.split()]


@pytest.mark.parametrize("m,n,k", [(5, 0, 24), (300, 0, 24), (0, 40, 24), (0, 0, 24), (0, 0, 0), (4, 0, 0)])
def test_empty_layers_need_no_scratch(m, n, k):
    none, gelu = _scratch(m, n, k)[:2]
    assert none == 0 and gelu == 0


@pytest.mark.parametrize("m,n,k", [(5, 40, 24), (3, 7, 0), (1, 1, 1), (1000, 100_000, 64)])
def test_scratch_holds_the_gradient_and_the_column_sums(m, n, k):
    none, gelu = _scratch(m, n, k)[:2]
    # at least one row of sums, and gz in 16 bits where an activation makes it
    assert none >= 4 * n
    assert gelu >= 4 * n + 2 * m * n
