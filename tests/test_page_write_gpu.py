"""The write of new keys and values into pages (fmha_page_write) on the GPU:
codes and scales are equal to the plain form's, since powers of two divide
exactly."""
import random

import pytest
import torch

from tests import cache_util as cu
from tests import page_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_attention_forward_02_gb300 import build, fmha
    build.build()
    fmha.lib()
    return fmha


def run(fm, k, v, slots, P, n_pages, seed=1, scales=None):
    """Writes into random pages; compares all of the cache."""
    g = torch.Generator().manual_seed(seed)
    H_k = k.shape[1]
    cache = [pu.draw_pages(g, n_pages, H_k, P) for _ in range(2)]
    if scales is not None:
        for _, s in cache:
            s.copy_(scales)
    dev = [(c.cuda(), s.cuda()) for c, s in cache]
    fm.page_write(k, v, torch.tensor(slots, dtype=torch.int32, device="cuda"), dev[0][0], dev[1][0], dev[0][1], dev[1][1])
    torch.cuda.synchronize()
    status = fm.device_status(reset=True)
    for (c, s), (dc, ds), x, name in zip(cache, dev, (k, v), "kv"):
        c = c.view(torch.uint8)
        pu.write(x.cpu(), slots, c, s)
        assert torch.equal(ds.cpu(), s), f"scales of {name}"
        got = dc.cpu().view(torch.uint8)
        bad = got != c
        assert not bad.any(), f"{int(bad.sum())} codes of {name}, first at {bad.nonzero()[0].tolist()}"
    return status


def seq_slots(P, lengths, news, seed):
    """Slots of each sequence's last `news` tokens in shuffled pages."""
    rng = random.Random(seed)
    pages = list(range(sum(pu.up(L, P) for L in lengths) + 2))
    rng.shuffle(pages)
    out = []
    for L, n in zip(lengths, news):
        own = [pages.pop() for _ in range(pu.up(L, P))]
        out += [own[i // P] * P + i % P for i in range(L - n, L)]
    return out, sum(pu.up(L, P) for L in lengths) + 2


CASES = {                                                 # dtype, P, H_k, lengths, news
    "one_token": ("bf16", 16, 1, [1], [1]),
    "decode": ("bf16", 64, 3, [64 * (i % 3) + 1 + (i * 29) % 64 for i in range(40)], [1] * 40),
    "few": ("f16", 32, 2, [32, 33, 40, 7, 64, 95], [9, 8, 10, 7, 33, 5]),
    "prompts": ("f16", 16, 2, [333, 16, 17, 1], [333, 16, 17, 1]),
    "chunks": ("bf16", 128, 2, [500, 129, 300], [450, 129, 45]),
    "large_page": ("bf16", 128, 1, [128, 127, 256], [128, 126, 129]),
    "across_chunks": ("f16", 64, 1, [64] * 9, [13] * 9),
}


@pytest.mark.parametrize("name", CASES)
def test_write(fm, name):
    dtype, P, H_k, lengths, news = CASES[name]
    g = torch.Generator().manual_seed(len(name))
    slots, n_pages = seq_slots(P, lengths, news, 3)
    N = len(slots)
    k, v = (cu.draw(g, (N, H_k, 128), dtype) * torch.exp(3 * torch.randn((N, H_k, 1), generator=g)).to(cu.DTYPES[dtype])
            for _ in range(2))
    assert run(fm, k.cuda(), v.cuda(), slots, P, n_pages) == 0


def test_strides_and_rows_that_are_not_written(fm):
    g = torch.Generator().manual_seed(2)
    rows = cu.draw(g, (70, 8 * 128 + 40), "bf16").cuda()
    k, v = rows[:, 16:16 + 256].unflatten(1, (2, 128)), rows[:, 512:768].unflatten(1, (2, 128))
    slots, n_pages = seq_slots(32, [50, 40], [40, 30], 5)
    for i in (0, 13, 39, 40, 69):
        slots[i] = -1 - i
    assert run(fm, k, v, slots, 32, n_pages) == 0
    heads_first = cu.draw(g, (2, 70, 128), "bf16").cuda().transpose(0, 1)
    assert run(fm, heads_first, k, slots, 32, n_pages) == 0
    assert run(fm, heads_first[:1].expand(70, 2, 128), k, slots, 32, n_pages) == 0


def test_extreme_values(fm):
    """Zeros, the smallest and largest values, infinities and NaN."""
    k = torch.randn((48, 2, 128), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    k[0] = 0.0
    k[1] *= 2.0 ** -120
    k[2] *= 2.0 ** 100
    k[3, 0, 5], k[4, 1, 6] = float("inf"), float("-inf")
    k[5, :, 7] = float("nan")
    k[6, 0] = float("nan")
    for i in range(10):                                   # the border between two exponents
        k[7 + i] = 448.0 * 2.0 ** (i - 5)
        k[17 + i] = 450.0 * 2.0 ** (i - 5)
    slots = [i * 16 for i in range(48)]
    assert run(fm, k.cuda(), k.flip(0).cuda(), slots, 16, 48) == 0


def test_any_scale_before(fm):
    """A page whose scale is not a power of two, zero or very large keeps it, or
    has its rows rounded to the larger one's steps."""
    g = torch.Generator().manual_seed(4)
    k = cu.draw(g, (32, 2, 128), "f16")
    scales = torch.ones((32, 2))
    scales[:8] = 2.0 ** -20
    scales[8:16] = 0.0
    scales[16:20] = 2.0 ** 50
    slots = [i * 64 + 9 for i in range(32)]
    assert run(fm, k.cuda(), k.cuda(), slots, 64, 32, scales=scales) == 0


def test_a_slot_outside_the_cache_is_reported(fm):
    k = cu.draw(torch.Generator().manual_seed(5), (20, 1, 128), "bf16").cuda()
    slots, n_pages = seq_slots(16, [20], [20], 6)
    slots[7] = n_pages * 16
    slots[8] = 0x7fffffff
    assert run(fm, k, k, slots, 16, n_pages) == fm.ERR_INVALID_ARG


def test_it_repeats(fm):
    """Twice the same write: the scales hold the values, so nothing changes."""
    g = torch.Generator().manual_seed(6)
    slots, n_pages = seq_slots(32, [60, 33], [25, 3], 7)
    k = cu.draw(g, (len(slots), 2, 128), "bf16").cuda()
    c, s = pu.draw_pages(g, n_pages, 2, 32)
    c, s, c2, s2 = c.cuda(), s.cuda(), c.cuda(), s.cuda()
    at = torch.tensor(slots, dtype=torch.int32, device="cuda")
    fm.page_write(k, k, at, c, c2, s, s2)
    once = c.view(torch.uint8).clone(), s.clone()
    fm.page_write(k, k, at, c, c2, s, s2)
    assert torch.equal(c.view(torch.uint8), once[0]) and torch.equal(s, once[1])
