"""Values past 32-bit offsets: O of drafts over the far entry of a large cache,
whose values have a mean and differ by head, dimension and place.  An entry of
zeros stands before it, so a load that wrapped would show."""
import pytest
import torch

from tests.test_cache_gpu import i32
from tests.test_tree_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2, 70], ids=["one_block", "two_blocks"])
def test_values_past_32_bits(fm, T):  # noqa: F811
    S, H_k, H, e = 1 << 22, 4, 8, 1                      # 2^31 elements an entry
    g = torch.Generator(device="cuda").manual_seed(53)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.empty((2, S, H_k, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[0].zero_()
    v[0].zero_()
    k[e].normal_(generator=g)
    place = (1 + torch.arange(S, device="cuda") / S)[:, None]
    for h in range(H_k):
        v[e, :, h] = ((1 + h + torch.arange(128, device="cuda") / 128) * place).to(torch.bfloat16)
    q, kn, vn = rnd(1, T, H, 128), rnd(1, T, H_k, 128), rnd(1, T, H_k, 128)
    L = S - 3
    o, lse = fm.tree_fwd(q, k, v, kn, vn, i32([L]), batch_idx=i32([e]))
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    rows = [0, T - 1]
    see = torch.arange(L + T, device="cuda")[None] <= L + torch.tensor(rows, device="cuda")[:, None]
    for h in range(H_k):
        keys, vals = (torch.cat([c[e, :L, h], n[0, :, h]]).double() for c, n in ((k, kn), (v, vn)))
        x = torch.einsum("thd,kd->thk", q[0, rows, 2 * h:2 * h + 2].double(), keys) * 128 ** -0.5
        x = x.masked_fill(~see[:, None, :], float("-inf"))
        w = torch.softmax(x, -1)
        want = torch.einsum("thk,kd->thd", w, vals)
        # every weight is rounded by up to 2^-8 of itself, O by as much, and sums of 2^22 in fp32 are cut over the
        # blocks (2^15 a block, so 2^-24 * 2^15 = 2^-9 at most, of either sum)
        tol = (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -8) * (torch.einsum("thk,kd->thd", w, vals.abs()) + want.abs()) / 2
        assert bool((want.abs() > 40 * tol).all())       # zeros, another head's or place's values would be seen
        assert bool(((o[0, rows, 2 * h:2 * h + 2].double() - want).abs() <= tol).all())
        assert bool(((lse[0, 2 * h:2 * h + 2][:, rows].T.double() - torch.logsumexp(x, -1)).abs() <= 1e-4).all())
