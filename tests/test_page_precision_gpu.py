"""How exact attention over a paged cache is where its output's own rounding
does not hide it: weights of keys whose values cancel, and small weights next to
a large one, against the formula in 64 bits."""
import pytest
import torch

from tests import cache_util as cu
from tests import page_util as pu
from tests import test_page_fwd_gpu as tf
from tests.test_page_fwd_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def exact(q, kc, ks, vc, vs, see, dtype):
    """One sequence and kv head in 64 bits, laid out as page_util.attend: O, LSE and the bounds on their errors."""
    scale = 128 ** -0.5
    keys = kc * ks[:, None]
    x = torch.einsum("tgd,kd->tgk", q, keys) * scale
    x = x.masked_fill(~see[:, None, :], -float("inf"))
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None]) * vs
    o = torch.einsum("tgk,kd->tgd", p, vc)
    seen = see[:, None, :].double()
    # a score: 128 products summed in fp32; elements of q off by 2^-21 of the row's largest; a few more fp32 roundings
    a = (torch.einsum("tgd,kd->tgk", q.abs(), keys.abs()) * scale * seen).amax(-1)
    ds = (a * 134 * 2.0 ** -23 + q.abs().amax(-1) * 2.0 ** -21 * (keys.abs().sum(-1) * seen).amax(-1) * scale +
          lse.abs() * 2.0 ** -21 + 1e-5)
    # a weight: f16's eleven bits (2^-11), then three terms of four bits (2^-12); and where the third term's steps
    # end, 2^-9 / 256 / 2, half a step, next to a largest one of 2^4: 2^-22
    ab = torch.einsum("tgk,kd->tgd", p, vc.abs())
    low = p.amax(-1, keepdim=True) * torch.einsum("tgk,kd->tgd", seen.expand(*p.shape), vc.abs())
    tol = ab * (2.0 ** -11 + 2.0 ** -12 + 2 * ds[..., None]) + low * 2.0 ** -22
    return o, lse, tol + (o.abs() + tol) * cu.HALF[dtype] + cu.SUBHALF[dtype], ds


def check(c, o, lse):
    o, lse, G, at = o.cpu(), lse.cpu(), c["H"] // c["H_k"], 0
    for b, (L, n) in enumerate(zip(c["L"], c["n"])):
        t, j = torch.arange(n)[:, None], torch.arange(L)[None]
        see = j <= L - n + t if c["mask"] == "causal" else torch.ones((n, L), dtype=torch.bool)
        for g in range(c["H_k"]):
            h = slice(g * G, (g + 1) * G)
            want, wl, tol, tl = exact(cu.f64(c["q"][at:at + n][:, h]), *tf.sequence(c, b, g, "k"), *tf.sequence(c, b, g, "v"), see, c["dtype"])
            cu.close(cu.f64(o[at:at + n][:, h]), want, tol, f"O of sequence {b} head {g}")
            cu.close(lse[at:at + n][:, h].double(), wl, tl, f"LSE of sequence {b} head {g}")
        at += n


# query heads, kv heads, tokens: units of 4, 8 and 16 rows, and of two groups of 16
SHAPES = [(8, 2, 1), (16, 2, 1), (32, 2, 1), (8, 2, 7)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,H_k,n", SHAPES)
def test_values_that_cancel(fm, H, H_k, n, dtype):  # noqa: F811
    """Two keys of nearly equal weight, the values of one the other's negatives."""
    B = 40
    c = tf.make(dtype, H, H_k, 16, [2] * B, [n] * B, mask="none", seed=H + n, q_scale=0.3)
    v = c["vc"].view(torch.uint8)
    v[:, :, 1] = v[:, :, 0] ^ 0x80
    o, lse, status = tf.run(fm, c)
    assert status == 0
    check(c, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,H_k,n", SHAPES)
def test_small_weights_beside_a_key_without_value(fm, H, H_k, n, dtype):  # noqa: F811
    """A key 2^18 above all others, whose value is zero: O is the others' alone."""
    B, L = 64, 1000
    c = tf.make(dtype, H, H_k, 64, [L] * B, [n] * B, mask="none", seed=3 + n, entries=[0] * B)
    g = torch.Generator().manual_seed(4)
    x = torch.rand(L, generator=g)                       # scores in log2 units: the keys' first dim
    x[3] = 18.0
    ids = c["table"][0, :pu.up(L, 64)].long()
    k = torch.zeros(len(ids) * 64, 128)
    k[:L, 0] = x
    codes = pu.codes(k.double()).view(-1, 64, 128)
    v = c["vc"].view(torch.uint8)
    v[ids] = torch.where(torch.arange(128) % 2 == 0, pu.codes(torch.tensor(40.0).double()), v[ids])   # a mean that does not cancel
    v[ids[0], :, 3] = 0
    cu.fill_nan(c["vc"], (ids[-1], slice(None), slice(L - (len(ids) - 1) * 64, None)))
    for h in range(H_k):
        c["kc"].view(torch.uint8)[ids, h] = codes
    c["ks"][ids] = 1.0
    c["vs"][ids] = 2.0 ** -6
    q = torch.zeros(B * n, H, 128)
    q[..., 0] = 0.6931471805599453 * 128 ** 0.5
    c["q"] = q.to(cu.DTYPES[dtype])
    o, lse, status = tf.run(fm, c)
    assert status == 0
    check(c, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_a_dim_of_q_above_the_others(fm, n, dtype):  # noqa: F811
    """One element of every row 2^9 times the others, on a dim where all keys are zero: the scores are the others'."""
    c = tf.make(dtype, 8, 2, 32, [300, 200], [n, n], seed=5, q_scale=0.2)
    g = torch.Generator().manual_seed(6)
    c["q"][..., 0] = 180.0
    c["q"][..., 1] = (0.125 + 0.125 * torch.rand(c["q"].shape[:-1], generator=g)).to(c["q"].dtype)
    k = c["kc"].view(torch.uint8)                        # keys: dim 1 alone, up to e4m3's largest
    nan = (k & 0x7F) == 0x7F
    k.copy_(torch.where(nan, k, 0))
    top = pu.codes(torch.rand(k.shape[:-1], generator=g).double() * 448)
    k[..., 1] = torch.where(nan[..., 1], k[..., 1], top)
    c["ks"].copy_(torch.where(c["ks"].isnan(), c["ks"], 1.0))
    o, lse, status = tf.run(fm, c)
    assert status == 0
    check(c, o, lse)
