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
