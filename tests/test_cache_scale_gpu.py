"""The smallest scales of the cache operators: every visible key has the same weight then."""
import pytest
import torch

from tests import cache_util as cu
from tests import test_cache_gpu as tc
from tests import test_tree_gpu as tt
from tests.test_tree_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
SCALES = [2.0 ** -126, 1e-38, 1e-40, 2.0 ** -149]        # fp32: the smallest normal, then subnormal ones


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype,T", [("bf16", 6), ("f16", 40), ("e4m3", 3)])
def test_tree_with_a_tiny_scale(fm, dtype, T, scale):  # noqa: F811
    c = tt.make(dtype, T, 8, 2, 300, [290, 3, 0], n_draft=[T, 1, T], seed=61)
    d, (o, lse) = tt.on_gpu(c), tt.outputs(c)
    fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse, scale=scale)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    tt.check(c, o, lse, scale=scale)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("Sq,mask", [(5, "causal"), (40, "none"), (40, "causal")])
def test_weights_with_a_tiny_scale(fm, Sq, mask, scale):  # noqa: F811
    S, seqlen = 300, [290, 41, 300]
    c = tc.make("bf16", Sq, 8, 2, S, seqlen, mask=mask, seed=62)
    c["lse"].fill_(0)
    for b, L in enumerate(seqlen):                       # each row: the logarithm of how many keys it sees
        t = torch.arange(Sq)
        c["lse"][b] = torch.log((t + L - Sq + 1 if mask == "causal" else torch.full((Sq,), L)).double()).float()
    acc = fm.cache_weights(c["q"].cuda(), c["kc"].cuda(), c["lse"].cuda(), tc.i32(seqlen), mask=mask, scale=scale)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    for b, L in enumerate(seqlen):
        see = torch.ones((Sq, L), dtype=torch.bool)
        if mask == "causal":
            see = see.tril(L - Sq)
        want = 4 * (see / see.sum(1, keepdim=True).double()).sum(0)      # 4 heads a group, every one alike
        # exp(-LSE): arguments below 8 and the LSE rounded a few times (2^-20 each), and 160 additions
        cu.close(acc[b, :, :L].cpu().double(), want.expand(2, L), want * (4 * 2.0 ** -20 + 164 * 2.0 ** -24), f"acc of sequence {b}")
        assert not bool(acc[b, :, L:].any())
