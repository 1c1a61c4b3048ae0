"""Attention over a paged e4m3 cache (fmha_page_fwd) on the GPU, against its
formula in 64 bits."""
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


def make(dtype, H, H_k, P, lengths, news=None, mask="causal", entries=None, seed=0, q_scale=2.0, extra_rows=0, lo=-8, hi=-4):
    """A case: news None is one row a sequence without cu_q.  Rows behind the
    lengths hold NaN, table entries behind them anything."""
    g, rng = torch.Generator().manual_seed(seed), random.Random(seed)
    B = len(lengths)
    entries = entries or rng.sample(range(B + 1), B)
    held = {}
    for b, L in enumerate(lengths):
        held[entries[b]] = max(held.get(entries[b], 0), pu.up(L, P))
    n_pages = sum(held.values()) + 2
    ids = rng.sample(range(n_pages), n_pages)
    width = max([1, *held.values()])
    table = [[rng.choice([-1, n_pages, 1 << 30]) for _ in range(width)] for _ in range(max(entries) + 1)]
    for e, n in held.items():
        for i in range(n):
            table[e][i] = ids.pop()
    c = dict(dtype=dtype, H=H, H_k=H_k, P=P, L=list(lengths), n=list(news) if news else [1] * B, entries=entries, mask=mask,
             has_cu=news is not None, table=torch.tensor(table, dtype=torch.int32))
    N = sum(c["n"]) + extra_rows
    c["q"] = cu.draw(g, (N, H, 128), dtype, q_scale)
    c["kc"], c["ks"] = pu.draw_pages(g, n_pages, H_k, P, lo, hi)
    c["vc"], c["vs"] = pu.draw_pages(g, n_pages, H_k, P, lo, hi)
    last = {}
    for b, L in enumerate(lengths):
        last[entries[b]] = max(last.get(entries[b], 0), L)
    live = set()
    for e, L in last.items():
        for i in range(pu.up(L, P)):
            live.add(table[e][i])
            cu.fill_nan(c["kc"], (table[e][i], slice(None), slice(max(0, L - i * P), None)))
            cu.fill_nan(c["vc"], (table[e][i], slice(None), slice(max(0, L - i * P), None)))
    for i in set(range(n_pages)) - live:
        cu.fill_nan(c["kc"], i)
        cu.fill_nan(c["vc"], i)
        c["ks"][i] = c["vs"][i] = float("nan")
    return c


def on_gpu(c):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cu_q = [0]
    for n in c["n"]:
        cu_q.append(cu_q[-1] + n)
    return dict(args=[c["q"].cuda(), c["kc"].cuda(), c["vc"].cuda(), c["ks"].cuda(), c["vs"].cuda(), c["table"].cuda(), i32(c["L"])],
                kw=dict(cu_q=i32(cu_q) if c["has_cu"] else None, max_q=max(1, *c["n"], 1), batch_idx=i32(c["entries"]),
                        mask=c["mask"]))


def outputs(c):
    N, H = c["q"].shape[:2]
    return cu.sentinel((N, H, 128), cu.DTYPES[c["dtype"]]), cu.sentinel((N, H), torch.float32)


def sequence(c, b, g, x):
    """Codes' values and scales of a sequence's rows."""
    ids = c["table"][c["entries"][b], :pu.up(c["L"][b], c["P"])].long()
    codes = pu.VALUES[c[x + "c"].view(torch.uint8)[ids, g].reshape(-1, 128).long()][:c["L"][b]]
    return codes, c[x + "s"][ids, g].double().repeat_interleave(c["P"])[:c["L"][b]]


def check(c, o, lse, scale=128 ** -0.5, out_scale=1.0, rows=None):
    o, lse = o.cpu(), lse.cpu()
    G, at = c["H"] // c["H_k"], 0
    chunk = max(c["n"]) * G > 32
    for b, (L, n) in enumerate(zip(c["L"], c["n"])):
        pick = torch.arange(n) if rows is None else torch.tensor(sorted({r for r in rows(n) if r < n}), dtype=torch.long)
        j, t = torch.arange(L), pick[:, None]
        see = (j[None] <= L - n + t) if c["mask"] == "causal" else torch.ones((len(pick), L), dtype=torch.bool)
        for g in range(c["H_k"]):
            h = slice(g * G, (g + 1) * G)
            want, wl, tol, tl = pu.attend(cu.f64(c["q"][at + pick][:, h]), *sequence(c, b, g, "k"), *sequence(c, b, g, "v"), see,
                                          scale, out_scale, c["dtype"], chunk)
            cu.close(cu.f64(o[at + pick][:, h]), want, tol, f"O of sequence {b} head {g}")
            cu.close(lse[at + pick][:, h].double(), wl, tl, f"LSE of sequence {b} head {g}")
        at += n
    assert cu.untouched(o[at:]) and cu.untouched(lse[at:]), "rows behind the last sequence"


def run(fm, c, **kw):
    d, (o, lse) = on_gpu(c), outputs(c)
    fm.page_fwd(*d["args"], **d["kw"], out=o, lse=lse, **kw)
    torch.cuda.synchronize()
    return o, lse, fm.device_status(reset=True)


CASES = {
    "one_key": dict(dtype="bf16", H=4, H_k=4, P=16, lengths=[1]),
    "empty": dict(dtype="bf16", H=8, H_k=2, P=16, lengths=[0, 5, 0]),
    "latency": dict(dtype="bf16", H=32, H_k=8, P=64, lengths=[1000]),
    "edges": dict(dtype="f16", H=8, H_k=2, P=32, lengths=[127, 128, 129, 31, 32, 33, 255, 256, 257]),
    "large_page": dict(dtype="bf16", H=8, H_k=1, P=128, lengths=[128, 129, 700]),
    "small_page": dict(dtype="f16", H=16, H_k=2, P=16, lengths=[15, 16, 17, 1111]),
    "group_16": dict(dtype="bf16", H=32, H_k=2, P=64, lengths=[513, 40]),
    "group_3": dict(dtype="f16", H=9, H_k=3, P=64, lengths=[300, 77]),
    "group_20": dict(dtype="bf16", H=40, H_k=2, P=64, lengths=[300, 77]),
    "group_65": dict(dtype="f16", H=65, H_k=1, P=64, lengths=[300, 7]),
    "group_128": dict(dtype="bf16", H=128, H_k=1, P=32, lengths=[1030]),
    "many": dict(dtype="bf16", H=8, H_k=2, P=64, lengths=[(i * 97) % 700 for i in range(90)]),
    "long": dict(dtype="f16", H=4, H_k=1, P=64, lengths=[20001]),
    "two_tokens": dict(dtype="bf16", H=8, H_k=2, P=64, lengths=[130, 2, 257], news=[2, 2, 1]),
    "few_tokens": dict(dtype="f16", H=8, H_k=2, P=32, lengths=[300, 7, 128, 64], news=[7, 7, 5, 1]),
    "some_have_none": dict(dtype="bf16", H=8, H_k=2, P=32, lengths=[300, 7, 128, 0], news=[0, 3, 0, 0], extra_rows=4),
    "prompt": dict(dtype="bf16", H=4, H_k=2, P=64, lengths=[500], news=[500]),
    "prompts": dict(dtype="f16", H=6, H_k=2, P=16, lengths=[333, 64, 1], news=[333, 64, 1], extra_rows=3),
    "chunks": dict(dtype="bf16", H=16, H_k=2, P=128, lengths=[900, 400, 128, 129], news=[150, 399, 100, 1]),
    "chunk_of_wide_groups": dict(dtype="bf16", H=96, H_k=1, P=64, lengths=[200], news=[33]),
    "mixed": dict(dtype="f16", H=12, H_k=4, P=64, lengths=[800, 500, 300, 64, 65, 1], news=[1, 130, 1, 64, 2, 1], extra_rows=1),
    "more_rows_than_keys": dict(dtype="bf16", H=4, H_k=2, P=32, lengths=[5, 0, 140], news=[20, 3, 300]),
    "all_keys": dict(dtype="bf16", H=8, H_k=2, P=32, lengths=[77, 300, 0], news=[90, 10, 2], mask="none"),
    "shared_rows": dict(dtype="bf16", H=8, H_k=2, P=32, lengths=[300, 300, 17], entries=[2, 2, 0]),
    "peaked": dict(dtype="bf16", H=8, H_k=2, P=64, lengths=[2999, 1500], q_scale=30.0),
    "flat": dict(dtype="f16", H=8, H_k=2, P=64, lengths=[2999], q_scale=2.0 ** -10),
    "scales_apart": dict(dtype="bf16", H=8, H_k=2, P=16, lengths=[777, 400], news=[3, 1], lo=-20, hi=4),
    "chunk_of_one_head": dict(dtype="bf16", H=2, H_k=2, P=16, lengths=[700, 300], news=[300, 257]),
    "chunk_of_half_units": dict(dtype="f16", H=8, H_k=2, P=32, lengths=[400, 130, 900], news=[31, 33, 97]),
    "chunk_scales_apart": dict(dtype="bf16", H=16, H_k=2, P=16, lengths=[777, 400], news=[70, 40], lo=-20, hi=4),
    "chunk_peaked": dict(dtype="f16", H=8, H_k=2, P=128, lengths=[1999], news=[140], q_scale=30.0),
    "chunk_and_tokens": dict(dtype="bf16", H=8, H_k=2, P=64, lengths=[900, 800, 700, 1], news=[120, 1, 1, 1]),
    "odd_rows_of_a_unit": dict(dtype="bf16", H=16, H_k=2, P=64, lengths=[600], news=[27]),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_the_formula(fm, name):
    c = make(seed=len(name), **CASES[name])
    o, lse, status = run(fm, c)
    assert status == 0
    check(c, o, lse)


@pytest.mark.parametrize("out_scale,scale", [(0.5, 0.3), (-2.0, 0.01), (0.0, 1.0)])
def test_scales_of_the_call(fm, out_scale, scale):
    c = make("bf16", 8, 2, 32, [400, 50], [3, 1], seed=3, q_scale=1.0)
    o, lse, status = run(fm, c, scale=scale, out_scale=out_scale)
    assert status == 0
    check(c, o, lse, scale, out_scale)


def test_scales_that_are_not_powers_of_two(fm):
    c = make("bf16", 8, 2, 32, [700, 129], seed=4)
    g = torch.Generator().manual_seed(5)
    for x in ("ks", "vs"):
        c[x] = c[x] * (0.5 + torch.rand(c[x].shape, generator=g))
    o, lse, status = run(fm, c)
    assert status == 0
    check(c, o, lse)


def test_pages_of_zeros(fm):
    """Pages whose values are all zero have the smallest scale, and their keys their weight."""
    c = make("bf16", 8, 2, 16, [600, 64], seed=6)
    ids = c["table"][c["entries"][0], :37].long()
    for i in ids[::2]:
        c["vc"].view(torch.uint8)[i] = 0
        c["vs"][i] = 2.0 ** -60
    for i in ids[1::4]:
        c["kc"].view(torch.uint8)[i] = 0
        c["ks"][i] = 2.0 ** -60
    o, lse, status = run(fm, c)
    assert status == 0
    check(c, o, lse)


@pytest.mark.parametrize("shape", ["sink", "rising", "falling", "steps"])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_small_weights_that_together_count(fm, shape, n):
    """A key far above thousands of equal ones, and scores that rise or fall over the context."""
    L, c = 16384, make("bf16", 16, 2, 64, [16384], [n], seed=7)
    x = torch.zeros(L)                                   # scores in log2 units
    if shape == "sink":
        x[3] = 14.0
    elif shape == "rising":
        x = torch.linspace(-30, 30, L)
    elif shape == "falling":
        x = torch.linspace(40, -10, L)
    else:
        x = ((torch.arange(L) // 777) % 5 * 9.0)
    # keys (x, 0, ..): the first dim holds the score, coarse in e4m3; the values are alike within pages
    ids = c["table"][c["entries"][0], :L // 64].long()
    k = torch.zeros(L, 128)
    k[:, 0] = x
    codes = pu.codes(k.double()).view(-1, 64, 128)
    for g in range(2):
        c["kc"].view(torch.uint8)[ids, g] = codes
        c["ks"][ids, g] = 1.0
        c["vs"][ids, g] = 2.0 ** -6
    v = c["vc"].view(torch.uint8)
    v[ids] = torch.where(torch.arange(128) % 2 == 0, pu.codes(torch.tensor(40.0).double()), v[ids])   # a mean that does not cancel
    q = torch.zeros(n, 16, 128)
    q[..., 0] = 0.6931471805599453 * 128 ** 0.5
    c["q"] = q.to(torch.bfloat16)
    o, lse, status = run(fm, c)
    assert status == 0
    check(c, o, lse)


@pytest.mark.parametrize("n", [4, 150])
def test_rows_that_are_not_finite(fm, n):
    c = make("bf16", 8, 2, 32, [300, 200], [n, 1], seed=8)
    c["q"][1, 3, 5] = float("nan")
    c["q"][2, 0, 7] = float("inf")
    o, lse, status = run(fm, c)
    bad = torch.zeros(n + 1, 8, dtype=torch.bool)
    bad[1, 3] = bad[2, 0] = True
    assert torch.equal(torch.isnan(o).any(-1).cpu(), bad) and torch.equal(torch.isnan(o).all(-1).cpu(), bad)
    assert torch.equal(torch.isnan(lse).cpu(), bad)
    c["q"][1, 3], c["q"][2, 0] = 0.0, 0.0
    o2, lse2, _ = run(fm, c)
    assert torch.equal(o.cpu()[~bad], o2.cpu()[~bad]) and torch.equal(lse.cpu()[~bad], lse2.cpu()[~bad])


@pytest.mark.parametrize("news", [None, [5, 30, 1], [200, 100, 77]])
def test_it_repeats_bit_for_bit(fm, news):
    c = make("bf16", 32, 8, 64, [5000, 3333, 1000], news, seed=9)
    o, lse, _ = run(fm, c)
    for _ in range(5):
        o2, lse2, _ = run(fm, c)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("k", [1, 40])
@pytest.mark.parametrize("what", ["length", "negative", "entry", "page", "rows", "order", "most"])
def test_values_outside_their_bounds_are_reported(fm, what, k):
    c = make("bf16", 8, 2, 32, [300, 200, 100], [2 * k, 3 * k, k], seed=10, entries=[0, 1, 2])
    d, (o, lse) = on_gpu(c), outputs(c)
    table, seqlen, cu_q, idx = d["args"][5], d["args"][6], d["kw"]["cu_q"], d["kw"]["batch_idx"]
    if what == "length":
        seqlen[1] = table.shape[1] * 32 + 1
        table[1] = table[1, 0]
    elif what == "negative":
        seqlen[1] = -7
    elif what == "entry":
        idx[1] = 3
    elif what == "page":
        table[1, 2] = c["kc"].shape[0]
    elif what == "rows":
        cu_q[3] = 1000
    elif what == "order":
        cu_q[2] = 1
    else:
        d["kw"]["max_q"] = 2 * k
    fm.page_fwd(*d["args"], **d["kw"], out=o, lse=lse)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG
    one = dict(c, L=[300], n=[2 * k], q=c["q"][:2 * k])  # the first sequence is served all the same
    check(one, o[:2 * k], lse[:2 * k])
    if what in ("negative", "entry"):
        assert bool((o[2 * k:5 * k] == 0).all())
    if what == "page":                                   # zeros for that page
        c["kc"].view(torch.uint8)[c["table"][1, 2].long()] = 0
        c["vc"].view(torch.uint8)[c["table"][1, 2].long()] = 0
        check(c, o, lse)


def test_random_cases(fm):
    rng = random.Random(11)
    for k in range(25):
        H, H_k = rng.choice([(8, 8), (8, 2), (16, 2), (12, 4), (6, 1), (33, 1)])
        B = rng.randint(1, 9)
        lengths = [rng.choice([0, 1, 64, 128, rng.randint(0, 1500)]) for _ in range(B)]
        news = None if rng.random() < 0.4 else [rng.choice([0, 1, 1, rng.randint(0, 9), rng.randint(0, 150)]) for _ in range(B)]
        if news is not None and sum(news) == 0:
            news[0] = 1
        c = make(rng.choice(["bf16", "f16"]), H, H_k, rng.choice([16, 32, 64, 128]), lengths, news, seed=k,
                 extra_rows=rng.randint(0, 2) if news else 0, mask=rng.choice(["causal", "causal", "none"]))
        o, lse, status = run(fm, c)
        assert status == 0
        check(c, o, lse)


@pytest.mark.parametrize("seed", range(12))
def test_random_chunks(fm, seed):
    """Sequences of many rows beside those of few, any group size, lengths around the
    tiles' ends, fewer keys than rows."""
    rng = random.Random(seed)
    for k in range(4):
        H_k = rng.choice([1, 2, 3, 4])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 33, 128 if H_k == 1 else 6])
        lengths, news = [], []
        for _ in range(rng.choice([1, 2, 3, 5])):
            n = min(rng.choice([0, 1, 3, 17, 33, 64, 100, 129, 200]), max(1, 600 // G))
            L = n + rng.choice([0, 0, 1, 15, 63, 64, 65, 127, 128, 129, 200, 500, 900, 1500])
            news.append(n)
            lengths.append(max(0, n - rng.choice([1, 3])) if rng.random() < 0.1 else L)
        if max(news) * G <= 32:
            news[0], lengths[0] = 33, 33 + rng.randint(0, 700)
        c = make(rng.choice(["bf16", "f16"]), H_k * G, H_k, rng.choice([16, 32, 64, 128]), lengths, news, seed=100 * seed + k,
                 mask=rng.choice(["causal", "causal", "none"]), extra_rows=rng.choice([0, 3]), q_scale=rng.choice([0.5, 2.0, 8.0]))
        o, lse, status = run(fm, c)
        assert status == 0
        check(c, o, lse)
