"""Attention of drafted trees where a few keys lie far above many others: the
many have small weights, which together count, and which the weights' rounding
to the tensors' type before P V must not lose.

O against its formula in 64 bits.  What is allowed: a weight is off by half a
step of its type, those in its subnormal range together by SMALL of their row's
sum (for e4m3 the reference is set again before more is lost; for fp16 each is
off by 2^-25 where the row's largest is 2^7 or more), and O's own rounding."""
import pytest
import torch

from tests import cache_util as cu
from tests.test_tree_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

L, H_K, G, B = 16384, 8, 8, 19               # 152 units that read one entry: a CTA goes through nearly a whole unit
SMALL = {"e4m3": 2.0 ** -5, "f16": L * 2.0 ** -32, "bf16": 0.0}


def scores(g, far):
    """Scores of kv head g's keys in nats, `far` times as far apart."""
    j = torch.arange(L, dtype=torch.float64)
    s = torch.zeros(L, dtype=torch.float64)
    if g == 0:                               # a sink
        s[0] = 10
    elif g == 1:
        s[0] = 12.5
    elif g == 2:                             # in the middle
        s[3001] = 11
    elif g == 3:                             # a sink, and a larger one later
        s[5], s[9000] = 9, 15
    elif g == 4:                             # every tile below the one before
        s = 12 - j * 0.01
    elif g == 5:                             # and above it
        s = j * 0.01
    elif g == 6:                             # nothing that counts for long, then keys that do
        s[:12000] = -60
        s[0], s[12000:] = 19, 9
    else:                                    # tiles of three heights
        s = -4.0 * ((j // 128) % 3)
        s[0] = 5
    return s * far


def make(dtype, T, far, seed):
    gen = torch.Generator().manual_seed(seed)
    q = torch.zeros(B, T, H_K * G, 128)
    q[..., 0] = 0.75 + torch.randint(0, 5, (B, T, H_K * G), generator=gen) / 8
    q[..., 1:3] = torch.randn((B, T, H_K * G, 2), generator=gen)
    k = torch.zeros(1, L, H_K, 128)
    k[0, :, :, 0] = torch.stack([scores(g, far) for g in range(H_K)], 1)
    k[..., 1:3] = 0.3 * torch.randn((1, L, H_K, 2), generator=gen)
    # a mean that is not zero, so that lost weights show
    v = 1 + torch.arange(128) / 128 + 0.25 * torch.randn((1, L, H_K, 128), generator=gen)
    v[0, :4, :, :] = 0
    kn, vn = torch.zeros(B, T, H_K, 128), torch.ones(B, T, H_K, 128)
    return [t.to(cu.DTYPES[dtype]) for t in (q, k, v, kn, vn)]


@pytest.mark.parametrize("T", [2, 20], ids=["one_block", "two_blocks"])
@pytest.mark.parametrize("dtype,far", [("e4m3", 1.0), ("e4m3", 0.8), ("f16", 1.6), ("f16", 1.3), ("bf16", 1.0)])
def test_many_small_weights_beside_a_large_one(fm, dtype, far, T):  # noqa: F811
    q, k, v, kn, vn = make(dtype, T, far, 3)
    i32 = lambda n, x: torch.full((n,), x, dtype=torch.int32, device="cuda")
    o, lse = fm.tree_fwd(*[t.cuda() for t in (q, k, v, kn, vn)], i32(B, L), batch_idx=i32(B, 0), scale=1.0)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    see = torch.cat([torch.ones((T, L), dtype=torch.bool), torch.ones((T, T), dtype=torch.bool).tril()], 1)
    for b in (0, B - 1):
        for g in range(H_K):
            keys, vals = (torch.cat([cu.f64(c[0, :, g]), cu.f64(n[b, :, g])]) for c, n in ((k, kn), (v, vn)))
            heads = slice(g * G, (g + 1) * G)
            want, wl, _, ds = cu.attend(cu.f64(q[b, :, heads]), keys, vals, see, 1.0, 1.0, dtype)
            x = torch.einsum("tgd,kd->tgk", cu.f64(q[b, :, heads]), keys).masked_fill(~see[:, None], -torch.inf)
            wabs = torch.einsum("tgk,kd->tgd", torch.exp(x - wl[..., None]), vals.abs())
            tol = wabs * (cu.HALF[dtype] + 2 * ds[..., None]) + SMALL[dtype] * vals.abs().amax(0)
            tol = tol + (want.abs() + tol) * cu.HALF[dtype] + cu.SUBHALF[dtype]
            cu.close(cu.f64(o[b, :, heads].cpu()), want, tol, f"O of sequence {b}, kv head {g}")
            cu.close(lse[b, heads].cpu().double().T, wl, ds, f"LSE of sequence {b}, kv head {g}")
