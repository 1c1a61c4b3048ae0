"""The cache operators on the default stream while another one is current: its handle is 0."""
import pytest
import torch

from tests import test_cache_gpu as tc
from tests import test_tree_gpu as tt
from tests.test_tree_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("default", [0, torch.cuda.default_stream], ids=["handle", "stream"])
def test_the_default_stream(fm, default):  # noqa: F811
    """The LSE, and the queries, are written there late: the calls come after that, not beside it."""
    stream = default if isinstance(default, int) else default()
    c = tc.make("bf16", 40, 8, 2, 900, [900, 301], mask="causal", seed=81)
    t = tt.make("bf16", 9, 8, 2, 900, [900, 301], seed=82)
    late, queries = c["lse"].cuda(), t["q"].cuda()
    args = c["q"].cuda(), c["kc"].cuda(), torch.zeros_like(late), tc.i32(c["seqlen"])
    acc, out = c["acc"].cuda(), torch.zeros(c["acc"].shape, device="cuda")
    d, (o, lse) = tt.on_gpu(t), tt.outputs(t)
    d["args"][0] = torch.zeros_like(queries)
    side = torch.cuda.Stream()
    fm.cache_weights(*args, mask="causal", acc=acc, out=out)      # the kernels are loaded before the streams part
    fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    args[2].copy_(late)
    d["args"][0].copy_(queries)
    with torch.cuda.stream(side):
        fm.cache_weights(*args, mask="causal", acc=acc, out=out, stream=stream)
        fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse, stream=stream)
    assert not torch.cuda.default_stream().query() and side.query()
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    tc.check_weights(c, out, torch.zeros_like(c["acc"]))
    tt.check(t, o, lse)
