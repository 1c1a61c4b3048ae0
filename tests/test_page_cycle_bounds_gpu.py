"""The paged-cache operators as a server runs them, with the bounds on O and LSE
that hold for units of every size."""
import pytest

from tests import page_util as pu
from tests import test_page_precision_gpu as tight
from tests.test_page_cycle_gpu import Server, fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_server_within_the_tight_bounds(fm, monkeypatch, dtype):  # noqa: F811
    def attend(q, kc, ks, vc, vs, see, scale, out_scale, dt, chunk):
        assert (scale, out_scale) == (128 ** -0.5, 1.0)
        return tight.exact(q, kc, ks, vc, vs, see, dt)

    monkeypatch.setattr(pu, "attend", attend)
    s = Server(fm, 4, 40, 12, dtype, seed=5)
    for n_new in ([50, 17, 0, 3], [1, 1, 1, 1], [4, 4, 0, 4], [-3, -2, 0, 0], [8, 1, 1, 7], [1, 0, 90, 1], [-48, 1, 1, 1], [9, 1, 1, 1],
                  [5, -20, 0, 1], [1, 60, 1, 1], [1, 1, 1, 1]):
        s.step(n_new)
