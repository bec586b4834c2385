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


def shared(n):
    """n rows, the first two of which begin with the same three pages; every page
    of the pool is in a row or on the stack."""
    rng = np.random.default_rng(n)
    case = PlanCase(rng, n, 16, 8, spare=40)
    case.held[:2] = [100, 70]
    need = ref.pages_for(case.held, 16)
    case.n_pages = int(need.sum()) - 3 + 40
    perm = rng.permutation(case.n_pages).astype(np.int32)
    case.table[:] = -7
    at = 0
    for s in range(n):
        k = 3 if s == 1 else 0
        case.table[s, :k] = case.table[0, :k]
        case.table[s, k:need[s]] = perm[at:at + need[s] - k]
        at += need[s] - k
    case.free = np.full(case.n_pages, -9, dtype=np.int32)
    case.n_free = case.n_pages - at
    case.free[:case.n_free] = perm[at:]
    return case


@pytest.mark.parametrize("n", [2, 40, 1500])
@pytest.mark.parametrize("ends", [[0], [1], [0, 1]])
@pytest.mark.parametrize("in_place", [True, False])
def test_a_page_of_two_rows_is_not_given_back(n, ends, in_place):
    case = shared(n)
    kv, q = case.held.copy(), np.zeros(n, dtype=np.int64)
    kv[ends] = 0
    got, code = case.call(kv, q, 5, in_place=in_place)
    unmoved(case, got, code, kv, q)


@pytest.mark.parametrize("n", [2, 40, 1500])
def test_rows_with_shared_pages_may_grow(n):
    case = shared(n)
    q = np.minimum(17, 8 * 16 - case.held)
    q[2:] = 0
    enough, code = case.check(case.held + q, q, int(q.sum()) + 3)
    assert enough and code == 0


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
