"""The write into pages (fmha_page_write) where runs of tokens are cut by slots
outside the cache: codes and scales equal to the plain form's."""
import pytest
import torch

from tests import cache_util as cu
from tests import page_util as pu
from tests.test_page_write_gpu import fm, seq_slots  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


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
