"""Block tables and slot maps (fmha_page_plan) on the GPU against the plain
form: whole numbers, so equal."""
import random

import pytest
import torch

from tests import page_util as pu

pytestmark = pytest.mark.gpu
KEPT = 0x3C3C3C3C


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_attention_forward_02_gb300 import build, fmha
    build.build()
    fmha.lib()
    return fmha


def make(seqlen, n_new, page, spare, width=None, rows=None, shuffle=True, seed=0):
    rng = random.Random(seed)
    B = len(seqlen)
    width = width or max(pu.up(max(L, L + n), page) for L, n in zip(seqlen, n_new)) + 1
    held = [pu.up(L, page) for L in seqlen]
    ids = list(range(sum(held) + spare + 2))
    rng.shuffle(ids)
    entry = list(range(B))
    if shuffle:
        rng.shuffle(entry)
    table, at = [[KEPT] * width for _ in range(B)], 0
    for b in range(B):
        for i in range(held[b]):
            table[entry[b]][i] = ids[at]
            at += 1
    free = ids[at:at + spare] + [KEPT] * (len(ids) - spare)
    rows = sum(max(0, n) for n in n_new) + 3 if rows is None else rows
    return dict(seqlen=seqlen, n_new=n_new, table=table, free_list=free, n_free=spare, page=page, rows=rows, entry=entry)


def on_gpu(c, in_place):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    a = dict(seqlen=i32(c["seqlen"]), n_new=i32(c["n_new"]), table=i32(c["table"]), free_list=i32(c["free_list"]),
             n_free=i32([c["n_free"]]))
    kw = dict(page_size=c["page"], max_tokens=c["rows"], batch_idx=i32(c["entry"]))
    if in_place:
        kw["new_seqlen"] = a["seqlen"]
    else:
        kw["n_free_out"] = i32([KEPT])
    return a, kw


def run_and_check(fm, c, in_place=False):
    a, kw = on_gpu(c, in_place)
    slots, pos, cu, new_len = fm.page_plan(**a, **kw)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    want = pu.plan(c["seqlen"], c["n_new"], c["table"], c["free_list"], c["n_free"], c["page"], c["rows"], c["entry"])
    assert slots.tolist() == want[0] and pos.tolist() == want[1]
    assert cu.tolist() == want[2] and new_len.tolist() == want[3]
    assert a["table"].tolist() == c["table"]
    n = want[4]
    assert (a["n_free"] if in_place else kw["n_free_out"]).tolist() == [n]
    assert a["free_list"].tolist() == c["free_list"]
    if not in_place:
        assert a["n_free"].tolist() == [c["n_free"]] and a["seqlen"].tolist() == c["seqlen"]
    return a, kw


CASES = {
    "one_new_request": dict(seqlen=[0], n_new=[1], page=16, spare=1),
    "one_token_fits": dict(seqlen=[15], n_new=[1], page=16, spare=0),
    "one_token_needs_a_page": dict(seqlen=[16], n_new=[1], page=16, spare=3),
    "nothing_to_do": dict(seqlen=[5, 0, 64], n_new=[0, 0, 0], page=64, spare=2),
    "ends": dict(seqlen=[5, 128, 129], n_new=[-5, -128, -129], page=128, spare=0),
    "drop_within_a_page": dict(seqlen=[20, 33], n_new=[-3, -1], page=32, spare=0),
    "given_back_and_taken": dict(seqlen=[100, 3, 0, 64], n_new=[-99, 70, 65, 1], page=32, spare=1),
    "too_few_pages": dict(seqlen=[16, 5, 32, 40, 7], n_new=[40, 1, 1, 3, 200], page=16, spare=4),
    "none_at_all": dict(seqlen=[0, 31, 64], n_new=[7, 1, 1], page=32, spare=0),
    "exactly_enough": dict(seqlen=[0, 0], n_new=[33, 32], page=32, spare=3),
    "cluster": dict(seqlen=[10, 5000, 77], n_new=[3333, -5000, 2000], page=16, spare=200),
    "decode_2000": dict(seqlen=[(i * 37) % 500 for i in range(2000)], n_new=[1] * 2000, page=64, spare=20),
    "most_sequences": dict(seqlen=[(i * 13) % 40 for i in range(8192)], n_new=[(i % 5) - 1 if (i * 13) % 40 else 1 for i in range(8192)],
                           page=16, spare=900),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_plan(fm, name, in_place):
    run_and_check(fm, make(**CASES[name]), in_place)


@pytest.mark.parametrize("seed", range(12))
def test_random_plans(fm, seed):
    rng = random.Random(seed)
    B, page = rng.choice([1, 2, 7, 31, 33, 300, 1025]), rng.choice([16, 32, 64, 128])
    seqlen = [rng.choice([0, page, rng.randint(0, 5 * page)]) for _ in range(B)]
    n_new = [rng.choice([0, 1, 1, 1, rng.randint(0, 4 * page), -rng.randint(0, L)]) for L in seqlen]
    run_and_check(fm, make(seqlen, n_new, page, rng.randint(0, 2 * B), seed=seed), bool(seed & 1))


def test_a_loop_of_steps_in_one_graph(fm):
    """Captured with everything in place and replayed: five decode steps."""
    page, c = 16, make([3, 15, 30, 0], [1, 1, 1, 1], 16, 6, width=8, rows=4)
    a, kw = on_gpu(c, True)
    outs = dict(slots=torch.empty(4, dtype=torch.int32, device="cuda"), positions=torch.empty(4, dtype=torch.int32, device="cuda"),
                cu_new=torch.empty(5, dtype=torch.int32, device="cuda"))
    kw.pop("max_tokens")
    keep = {k: v.clone() for k, v in a.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fm.page_plan(**a, **kw, **outs)
    torch.cuda.current_stream().wait_stream(s)
    for k, v in keep.items():
        a[k].copy_(v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fm.page_plan(**a, **kw, **outs)
    L, n = c["seqlen"], c["n_free"]
    for _ in range(5):
        g.replay()
        want = pu.plan(L, c["n_new"], c["table"], c["free_list"], n, page, 4, c["entry"])
        L, n = want[3], want[4]
        assert outs["slots"].tolist() == want[0] and outs["positions"].tolist() == want[1]
        assert a["seqlen"].tolist() == L and a["n_free"].tolist() == [n] and a["table"].tolist() == c["table"]
    assert fm.device_status(reset=True) == 0


@pytest.mark.parametrize("what", ["length", "negative", "drop", "entry", "rows", "too_long", "free", "page"])
def test_values_outside_their_bounds_are_reported(fm, what):
    c = make([40, 20, 7], [1, 1, 1], 16, 2, width=3, shuffle=False)
    if what == "length":
        c["seqlen"][1] = 49
    elif what == "negative":
        c["seqlen"][1] = -1
    elif what == "drop":
        c["n_new"][1] = -21
    elif what == "entry":
        c["entry"][1] = 3
    elif what == "rows":
        c["rows"] = 2
    elif what == "too_long":
        c["n_new"][0] = 9
    elif what == "free":
        c["n_free"] = 100
    else:
        c["table"][1][1] = 1000
    a, kw = on_gpu(c, False)
    slots, pos, cu, new_len = fm.page_plan(**a, **kw)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG
    # the others are served all the same
    assert pos[0].item() == 40
    if what != "too_long":
        assert slots[0].item() == c["table"][0][2] * 16 + 8 and new_len[0].item() == 41
    else:
        assert slots.tolist() == [-1] * 6 and cu.tolist() == [0, 6, 6, 6] and new_len.tolist() == [40, 21, 8]
    if what == "rows":
        assert cu.tolist() == [0, 1, 2, 2]
    if what == "page":
        assert slots[1].item() == -1
    if what == "entry":
        assert slots[1].item() == -1 and new_len.tolist() == [41, 20, 8]
    if what == "drop":
        assert new_len.tolist() == [41, 0, 8]


def test_as_many_rows_as_32_bits_count(fm):
    """The rows behind the last token, up to the largest N, are told so too."""
    n = 2 ** 31 - 1
    c = make([5, 0], [2, 1], 16, 3, shuffle=False)
    a, _ = on_gpu(c, False)
    slots, pos, cu, new_len = fm.page_plan(**a, page_size=16, max_tokens=n)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    page = c["table"][0][0] * 16
    assert pos[:4].tolist() == [5, 6, 0, -1] and slots[:2].tolist() == [page + 5, page + 6] and cu.tolist() == [0, 2, 3]
    assert new_len.tolist() == [7, 1]
    for x in (slots, pos):
        assert bool((x[3:n // 2] == -1).all()) and bool((x[n // 2:] == -1).all())
