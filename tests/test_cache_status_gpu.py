"""fmha_device_status: what it says of work on streams that do not wait for the
default one, and after errors of several operators."""
import pytest
import torch

from tests import test_tree_gpu as tt
from tests.test_tree_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_status_covers_work_on_every_stream(fm):  # noqa: F811
    """A length outside its bounds, met by a kernel that has not begun yet: the call synchronises the device."""
    c = tt.make("bf16", 4, 8, 2, 200, [100, 50], seed=91)
    d, (o, lse) = tt.on_gpu(c), tt.outputs(c)
    fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse)
    d["args"][5] = torch.tensor([201, 50], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse)
    assert not side.query()
    assert fm.device_status() == fm.ERR_INVALID_ARG and side.query()
    assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG    # the call before left it
    assert fm.device_status() == 0
