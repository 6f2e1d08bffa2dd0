"""The tolerances of the orthogonalised update, from a model of its roundings."""
import numpy as np
import pytest

from oracle import update_oracle as U
from tests import update_model as R


def errors(case, **kw):
    # (of many small matrices all, of large ones one or two)
    g = R.gradients(case, min(case.count, max(1, 300_000 // (case.rows * case.cols))))
    want = np.stack([U.orthogonalize(m, case.steps) for m in g])
    return R.relative(np.stack([R.modelled(m, case.steps, case.pair, **kw) for m in g]), want)


@pytest.mark.parametrize("case", R.CASES, ids=lambda c: c.name)
def test_bounds_follow_from_the_roundings(case):
    e = errors(case)
    assert case.bound / 1.4 <= e <= case.bound / 1.1, e


@pytest.mark.parametrize("case", [c for c in R.CASES if c.rank < min(c.rows, c.cols) <= 400
                                  and c.count * c.rows * c.cols < 4_000_000], ids=lambda c: c.name)
def test_bounds_reject_the_low_part_by_the_diagonal(case):
    assert errors(case, low_by_diagonal=True) > case.bound


@pytest.mark.parametrize("case", [R.CASES[0], R.CASES[2]], ids=lambda c: c.name)
def test_bounds_reject_two_steps_without_a_low_part(case):
    assert errors(case, lows=2) > case.bound


def test_output_rounding_alone():
    x = np.random.default_rng(1).normal(size=(400, 400)).astype(np.float32)
    assert abs(R.relative(R.to_bf16(x), x) - 1.66e-3) < 0.03e-3
