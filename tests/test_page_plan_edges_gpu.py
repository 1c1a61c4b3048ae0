"""Plans (fmha_page_plan) at the edges of what they are given: pages that are none, no sequences."""
import pytest
import torch

from tests import test_page_plan_gpu as tp
from tests.test_page_plan_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [-1, 1000])
@pytest.mark.parametrize("n_new", [-20, -5])
def test_a_page_outside_the_cache_that_is_given_back_is_reported(fm, page, n_new):  # noqa: F811
    """Not only once a later call hands it out."""
    c = tp.make([40, 20, 7], [1, n_new, 1], 16, 2, width=3, shuffle=False)
    c["table"][1][1] = page
    a, kw = tp.on_gpu(c, False)
    fm.page_plan(**a, **kw)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG


@pytest.mark.parametrize("rows", [0, 5])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_step_without_sequences(fm, rows, in_place):  # noqa: F811
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    kept = tp.KEPT
    given = dict(slots=i32([kept] * rows), positions=i32([kept] * rows), cu_new=i32([kept]), new_seqlen=i32([]))
    table, free, n_free, n_free_out = i32([[3, 1]]), i32([0, 2]), i32([2]), i32([kept])
    got = fm.page_plan(i32([]), i32([]), table, free, n_free, page_size=16, **given, **({} if in_place else dict(n_free_out=n_free_out)))
    fresh = fm.page_plan(i32([]), i32([]), table, free, n_free, page_size=16, max_tokens=rows)
    for out in (got, fresh):
        assert [x.tolist() for x in out] == [[-1] * rows, [-1] * rows, [0], []]
    assert n_free.tolist() == [2] and n_free_out.tolist() == [kept if in_place else 2]
    assert table.tolist() == [[3, 1]] and free.tolist() == [0, 2] and fm.device_status(reset=True) == 0


def test_a_step_of_drops_alone(fm):  # noqa: F811
    tp.run_and_check(fm, tp.make([40, 20], [-9, -20], 16, 1, rows=0))


def test_sequences_that_share_their_first_pages(fm):  # noqa: F811
    """The first to end drops what lies behind them, the last all: every page comes back once."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, free, n_free = i32([[4, 2, 5, 0], [4, 2, 1, -1]]), i32([3] + [-1] * 5), i32([1])
    seqlen = i32([60, 40])
    step = lambda n: fm.page_plan(seqlen, i32(n), table, free, n_free, page_size=16, max_tokens=4, new_seqlen=seqlen)
    step([-28, 1])                                       # 32 tokens in the shared pages
    assert seqlen.tolist() == [32, 41] and n_free.tolist() == [3] and free[:3].tolist() == [3, 5, 0]
    seqlen[0] = 0                                        # it has ended: the pages are the other's alone
    step([0, -41])
    assert seqlen.tolist() == [0, 0] and n_free.tolist() == [6] and sorted(free.tolist()) == list(range(6))
    assert fm.device_status(reset=True) == 0
