"""The write into pages (fmha_page_write) where runs of tokens are cut by slots
outside the cache, and where a page's scale is no power of two: codes and
scales equal to the plain form's."""
from fractions import Fraction

import pytest
import torch

from tests import cache_util as cu
from tests import page_util as pu
from tests.test_page_write_gpu import fm, seq_slots  # noqa: F401  (the fixture)



def run(fm, k, v, slots, P, n_pages, scales, seed=1):  # noqa: F811
    """Writes into random pages with the scales [n_pages, H_k] before; compares all of the cache.
    A slot outside the cache is to the plain form a token that is not written."""
    g = torch.Generator().manual_seed(seed)
    cache = [pu.draw_pages(g, n_pages, k.shape[1], P) for _ in range(2)]
    for _, s in cache:
        s.copy_(scales)
    (kc, ks), (vc, vs) = dev = [(c.cuda(), s.cuda()) for c, s in cache]
    fm.page_write(k.cuda(), v.cuda(), torch.tensor(slots, dtype=torch.int32, device="cuda"), kc, vc, ks, vs)
    torch.cuda.synchronize()
    status = fm.device_status(reset=True)
    inside = [s if 0 <= s < n_pages * P else -1 for s in slots]
    for (c, s), (dc, ds), x, name in zip(cache, dev, (k, v), "kv"):
        c = c.view(torch.uint8)
        pu.write(x, inside, c, s)
        assert torch.equal(ds.cpu(), s), f"scales of {name}"
        bad = dc.cpu().view(torch.uint8) != c
        assert not bad.any(), f"{int(bad.sum())} codes of {name}, first at {bad.nonzero()[0].tolist()}"
    return status


# page size; the sequence's tokens, and the last of them that are new; which of these have a slot outside the cache
RUNS = {
    "short": (16, 20, 20, [7, 8]),
    "behind_cached_rows": (16, 30, 25, [3, 4, 13]),
    "at_both_ends": (32, 32, 32, [0, 1, 31]),
    "long": (128, 128, 128, [0, 15, 16, 40, 41, 42, 127]),
    "long_behind_cached_rows": (64, 200, 150, [0, 20, 21, 70, 149]),
    "a_whole_chunk": (64, 64, 64, list(range(10, 45))),
}


@pytest.mark.gpu
@pytest.mark.parametrize("before", [2.0 ** -20, 2.0 ** -7, 2.0 ** 4])
@pytest.mark.parametrize("name", RUNS)
def test_slots_outside_the_cache_within_a_run(fm, name, before):  # noqa: F811
    """The tokens around them are one run, whatever the page's scale was: larger than theirs, smaller or equal."""
    P, L, n, out = RUNS[name]
    g = torch.Generator().manual_seed(len(name))
    k, v = (cu.draw(g, (n, 5, 128), "bf16") * torch.exp(2 * torch.randn((n, 5, 1), generator=g)).to(torch.bfloat16) for _ in range(2))
    slots, n_pages = seq_slots(P, [L], [n], 4)
    for i, j in enumerate(out):
        slots[j] = (n_pages * P, 0x7fffffff, -1)[i % 3]
    assert run(fm, k, v, slots, P, n_pages, torch.full((n_pages, 5), before)) == fm.ERR_INVALID_ARG


LEVELS = [pu.VALUES[c].item() for c in range(127)]       # of the codes 0 .. 0x7E, ascending


def nearest(x):
    """e4m3 code of a whole fraction, to nearest even, saturating."""
    a, lo, hi = abs(x), 0, 126
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if Fraction(LEVELS[mid]) <= a else (lo, mid)
    below, above = a - Fraction(LEVELS[lo]), Fraction(LEVELS[hi]) - a
    c = hi if above < below or (above == below and hi % 2 == 0) else lo
    return c | (0x80 if x < 0 else 0)


def test_nearest_is_the_types_rounding():
    x = torch.cat([torch.randn(400, generator=torch.Generator().manual_seed(1)) * 2.0 ** torch.randint(-12, 10, (400,)),
                   (pu.VALUES[:126] + pu.VALUES[1:127]).float() / 2])
    assert [nearest(Fraction(v)) & 0x7F for v in x.tolist()] == (pu.codes(x.double()) & 0x7F).tolist()


def ties(gen, scale, n, dtype, most=126):
    """n values, of which many are halfway between two codes times the scale, or a step of the type beside that."""
    code = torch.randint(0, most, (n,), generator=gen)
    half = (pu.VALUES[code] + pu.VALUES[code + 1]) / 2 * scale
    x = half.to(cu.DTYPES[dtype])
    step = torch.randint(-1, 2, (n,), generator=gen).to(torch.int16)
    x = (x.view(torch.int16) + step * (x.view(torch.int16) > 1)).view(x.dtype)
    return torch.where(torch.rand(n, generator=gen) < 0.5, -x, x)


@pytest.mark.gpu
@pytest.mark.parametrize("most", [126, 116])             # largest code: with the first, some scales have to grow
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("P,n", [(16, 1), (16, 9), (128, 90)])
def test_new_rows_over_a_scale_that_is_no_power_of_two(fm, P, n, dtype, most):  # noqa: F811
    """Quotients, and products where the scale grows, are rounded once, ties to even."""
    scales, n_pages = [1.5, 1.25, 3.0 * 2.0 ** -9, 1.0 + 2.0 ** -23, 0.7, 2.0 - 2.0 ** -23, 448.0 / 127], 14
    s = torch.tensor(scales).repeat(2)[:, None].expand(n_pages, 2).contiguous()
    g = torch.Generator().manual_seed(P + n)
    x = torch.stack([torch.stack([ties(g, s[p, 0].double(), n * 128, dtype, most).view(n, 128) for _ in range(2)], 1) for p in range(n_pages)])
    slots = [p * P + 5 + i for p in range(n_pages) for i in range(n)]
    c, _ = pu.draw_pages(g, n_pages, 2, P)
    kc, vc, ks, vs = c.cuda(), c.cuda(), s.cuda(), s.cuda()
    k = x.flatten(0, 1).contiguous()
    fm.page_write(k.cuda(), k.flip(1).contiguous().cuda(), torch.tensor(slots, dtype=torch.int32, device="cuda"), kc, vc, ks, vs)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    want, kept = c.view(torch.uint8).clone(), 0
    for p in range(n_pages):
        for h in range(2):
            old = Fraction(s[p, h].item())
            new = max(old, Fraction(2.0 ** pu.exponent(x[p, :, h].double().abs().max().item())))
            assert ks[p, h].item() == float(new) and vs[p, 1 - h].item() == float(new)
            kept += new == old
            want[p, h, 5:5 + n] = torch.tensor([nearest(Fraction(v) / new) for v in x[p, :, h].double().flatten().tolist()],
                                               dtype=torch.uint8).view(n, 128)
            if new > old:
                again = torch.tensor([nearest(Fraction(LEVELS[v]) * old / new) for v in range(127)], dtype=torch.uint8)
                before = want[p, h, :5].long()
                want[p, h, :5] = again[before & 0x7F] | (before & 0x80).to(torch.uint8)
    assert kept >= (n_pages * 2 if most == 116 else 4)
    zero = lambda t: torch.where(t == 0x80, 0, t)        # zeros of either sign
    got = kc.cpu().view(torch.uint8)
    bad = zero(got) != zero(want)
    assert not bad.any(), f"{int(bad.sum())} codes, first at {bad.nonzero()[0].tolist()}"
    assert torch.equal(zero(vc.cpu().view(torch.uint8)[:, :, 5:5 + n].flip(1)), zero(got[:, :, 5:5 + n]))


@pytest.mark.gpu
@pytest.mark.parametrize("P,n", [(16, 1), (128, 40)])
def test_rows_before_under_a_scale_that_was_no_power_of_two(fm, P, n):  # noqa: F811
    """The scale grows to a power of two, and the cached codes' products are rounded once."""
    g = torch.Generator().manual_seed(7)
    n_pages, off = 256, 7
    c = torch.randint(0, 126, (n_pages, 1, P, 128), generator=g).to(torch.uint8)
    # old scales for which a code's product lies a little beside the middle of two: code * (old / new) = (a + b) / 2 * (1 +- 2^-24)
    a, b = torch.randint(8, 118, (2, n_pages), generator=g)
    old = ((pu.VALUES[a] + pu.VALUES[a + 1]) / 2 / pu.VALUES[b + 1]).float()
    old = (old.view(torch.int32) + torch.randint(-1, 2, (n_pages,), generator=g).to(torch.int32)).view(torch.float32)
    new = torch.exp2(torch.ceil(torch.log2(old)) + 1)
    old, s = old[:, None], new[:, None]
    c[:, 0, 0, :] = (b + 1)[:, None].to(torch.uint8)
    x = torch.randn((n_pages * n, 1, 128), generator=g).clamp(-1, 1).to(torch.bfloat16)
    x = x.view(n_pages, n, 128) * s[:, :, None].to(torch.bfloat16)
    x[:, 0, 0] = 448 * s[:, 0].to(torch.bfloat16)        # the run's largest sets the new scale
    slots = [p * P + off + i for p in range(n_pages) for i in range(n)]
    k = x.reshape(-1, 1, 128).contiguous().cuda()
    kc, vc = (c.cuda().view(pu.E4M3).clone() for _ in range(2))
    ks, vs = old.cuda(), old.cuda()
    fm.page_write(k, k, torch.tensor(slots, dtype=torch.int32, device="cuda"), kc, vc, ks, vs)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0 and torch.equal(ks.cpu(), s)
    got = kc.cpu().view(torch.uint8)[:, 0, :off]
    for p in range(n_pages):
        f = Fraction(old[p, 0].item()) / Fraction(s[p, 0].item())
        again = torch.tensor([nearest(Fraction(LEVELS[v]) * f) for v in range(127)], dtype=torch.uint8)
        assert torch.equal(got[p], again[c[p, 0, :off].long()]), f"page {p}"


@pytest.mark.gpu
def test_strides_that_are_never_stepped_along(fm):  # noqa: F811
    """One token, or one head: its stride may be anything."""
    x = cu.draw(torch.Generator().manual_seed(8), (4096,), "bf16")
    one_token, one_head = x.as_strided((1, 3, 128), (1001, 136, 1)), x.as_strided((5, 1, 128), (264, 77, 1))
    for k, slots in ((one_token, [3]), (one_head, [16, 17, 18, 30, 31])):
        dev = x.cuda().as_strided(k.shape, k.stride())   # cuda() of the view itself would be packed
        c, s = pu.draw_pages(torch.Generator().manual_seed(9), 2, k.shape[1], 16)
        kc, vc, ks, vs = c.cuda(), c.cuda(), s.cuda(), s.cuda()
        fm.page_write(dev, dev, torch.tensor(slots, dtype=torch.int32, device="cuda"), kc, vc, ks, vs)
        torch.cuda.synchronize()
        assert fm.device_status(reset=True) == 0
        c = c.view(torch.uint8)
        pu.write(k, slots, c, s)
        for got, scale in ((kc, ks), (vc, vs)):
            assert torch.equal(got.cpu().view(torch.uint8), c) and torch.equal(scale.cpu(), s)
