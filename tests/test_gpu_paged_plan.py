"""GPU tests of the page plan on tables and stacks that it must leave alone."""
import numpy as np
import pytest

import paged_util as ref
from test_gpu_paged import PlanCase, _lib  # noqa: F401 (_lib: the module's fixture)

pytestmark = pytest.mark.gpu


def unmoved(case, got, code, kv, q):
    """The error word is set and nothing has moved; the offsets are written."""
    assert code == 2
    assert np.array_equal(got["table"], case.table) and np.array_equal(got["free"], case.free)
    assert got["n_free"] == case.n_free and (got["slots"] == -1).all()
    assert np.array_equal(got["row_off"], np.concatenate([[0], np.cumsum(kv)]))
    assert np.array_equal(got["q_off"], np.concatenate([[0], np.cumsum(q)]))


@pytest.mark.parametrize("n", [12, 1500])
@pytest.mark.parametrize("height", ["negative", "above the pool"])
@pytest.mark.parametrize("in_place", [True, False])
def test_a_bad_stack_height_moves_nothing(n, height, in_place):
    rng = np.random.default_rng(3)
    case = PlanCase(rng, n, 16, 6, spare=60)
    case.n_free = -1 if height == "negative" else case.n_pages + 1
    kv = rng.integers(0, 6 * 16 + 1, n)                 # some grow, some shrink
    q = np.minimum(kv, 3)
    got, code = case.call(kv, q, int(q.sum()) + 2, in_place=in_place)
    unmoved(case, got, code, kv, q)
