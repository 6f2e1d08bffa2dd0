"""The orthogonalised update's error against 64 bits on the GPU: rank-deficient
and full gradients, small and large, held to what its roundings leave (the
bounds of tests/update_model.py)."""
import numpy as np
import pytest
import torch

from oracle import update_oracle as U
from tests import update_model as R
from tests.gpu_common import say, to_f64
from tests.test_gpu_update import DT, dev, orth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", R.CASES, ids=lambda c: c.name)
def test_error_against_64_bits(case):
    say(f"orthogonalize {case.name}")
    g = R.gradients(case)
    out = to_f64(orth(dev(g, DT[case.dtype]), steps=case.steps))
    some = range(case.count) if g.size <= 1 << 20 else (0, case.count - 1)
    want = np.stack([U.orthogonalize(g[i], case.steps) for i in some])
    e = R.relative(out[list(some)], want)
    say(f"rel {e:.2e}, bound {case.bound:.2e}")
    assert e <= case.bound
