"""Accumulated attention weight of cached keys (fmha_cache_weights) and
eviction by it (fmha_cache_evict), on the GPU: against their formulas, and a
decode loop that uses them with generation and drafted trees."""
import math

import pytest
import torch

from tests import cache_util as cu

pytestmark = pytest.mark.gpu
i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_attention_forward_02_gb300 import build, fmha
    build.build()
    fmha.lib()
    return fmha


# ---------------------------------------------------------------------------
# Weights
# ---------------------------------------------------------------------------

def make(dtype, Sq, H, H_k, S_max, seqlen, n_query=None, mask="none", batch_idx=None, seed=0):
    """Inputs with the LSE of their own visible keys (-inf for rows without any)."""
    g = torch.Generator().manual_seed(seed)
    B = len(seqlen)
    Bc = B if batch_idx is None else max(batch_idx) + 1
    c = dict(dtype=dtype, B=B, Sq=Sq, H=H, H_k=H_k, seqlen=seqlen, n=n_query or [Sq] * B, mask=mask,
             entry=batch_idx or list(range(B)), n_query=n_query, batch_idx=batch_idx)
    c["q"] = cu.draw(g, (B, Sq, H, 128), dtype, 2.0)
    c["kc"] = cu.draw(g, (Bc, S_max, H_k, 128), dtype)
    c["acc"] = torch.rand((Bc, H_k, S_max), generator=g)
    c["lse"] = torch.full((B, H, Sq), math.nan)               # rows that are no queries
    c["want"], c["tol"] = c["acc"].double().clone(), torch.zeros_like(c["acc"]).double()
    G = H // H_k
    for b in range(B):
        L, n, e = seqlen[b], c["n"][b], c["entry"][b]
        see = torch.ones((n, L), dtype=torch.bool)
        if mask == "causal":
            see = see.tril(L - n)
        for gg in range(H_k):
            keys = cu.f64(c["kc"][e, :L, gg])
            q = cu.f64(c["q"][b, :n, gg * G:(gg + 1) * G])
            x = (torch.einsum("tgd,kd->tgk", q, keys) * 128 ** -0.5).masked_fill(~see[:, None, :], -math.inf)
            lse = torch.logsumexp(x, -1).float() if L else torch.full((n, G), -math.inf)
            c["lse"][b, gg * G:(gg + 1) * G, :n] = lse.T
            w = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse).double()[..., None])
            c["want"][e, gg, :L] += w.sum((0, 1))
            # a score is 128 products summed in fp32 (2^-23 of the sum of their
            # magnitudes an addition), the exponent's argument and the
            # exponential round a few times, and the sum over rows n * G times
            a = torch.einsum("tgd,kd->tgk", q.abs(), keys.abs()) * 128 ** -0.5
            rel = (a * 130 + 16 * lse.abs().nan_to_num(0, 0, 0)[..., None]) * 2.0 ** -23 + 2.0 ** -20
            c["tol"][e, gg, :L] += (w * rel).sum((0, 1))
        c["tol"][e, :, :L] += c["want"][e, :, :L] * (n * G + 4) * 2.0 ** -24
        cu.fill_nan(c["q"], (b, slice(n, None)))
        cu.fill_nan(c["kc"], (e, slice(L, None)))
    return c


def weights(fm, c, **kw):
    return fm.cache_weights(c["q"].cuda(), c["kc"].cuda(), c["lse"].cuda(), i32(c["seqlen"]), n_query=i32(c["n_query"]),
                            batch_idx=i32(c["batch_idx"]), mask=c["mask"], **kw)


def check_weights(c, got, was):
    """Rows below each length hold the sum, all others what they held before."""
    got = got.cpu().double()
    want, tol = was.double().clone(), torch.zeros_like(c["tol"])
    for e, L in zip(c["entry"], c["seqlen"]):
        want[e, :, :L], tol[e, :, :L] = c["want"][e, :, :L], c["tol"][e, :, :L]
    cu.close(got, want, tol, "acc")


W_CASES = {
    "decode": dict(dtype="bf16", Sq=1, H=32, H_k=8, S_max=1000, seqlen=[1000, 0, 1, 129, 256, 257]),
    "decode_e4m3": dict(dtype="e4m3", Sq=1, H=12, H_k=4, S_max=700, seqlen=[700, 513], batch_idx=[2, 0]),
    "one_head_group": dict(dtype="f16", Sq=1, H=128, H_k=1, S_max=300, seqlen=[300]),
    "window": dict(dtype="bf16", Sq=33, H=16, H_k=2, S_max=900, seqlen=[900, 33, 640], mask="causal"),
    "window_no_mask": dict(dtype="e4m3", Sq=40, H=16, H_k=2, S_max=600, seqlen=[600, 1, 255], n_query=[40, 3, 17]),
    "prompt": dict(dtype="bf16", Sq=1200, H=6, H_k=2, S_max=1200, seqlen=[1200], mask="causal"),
    "prompt_ragged": dict(dtype="f16", Sq=700, H=4, H_k=4, S_max=800, seqlen=[700, 300, 0, 513],
                          n_query=[700, 300, 0, 512], mask="causal", batch_idx=[3, 1, 0, 2]),
    "more_queries_than_keys": dict(dtype="bf16", Sq=300, H=4, H_k=2, S_max=200, seqlen=[200, 70], mask="causal"),
    "no_queries": dict(dtype="bf16", Sq=5, H=4, H_k=2, S_max=600, seqlen=[600, 300], n_query=[0, 5]),
    "long": dict(dtype="bf16", Sq=150, H=8, H_k=1, S_max=9000, seqlen=[8999], mask="causal"),
    "odd_group": dict(dtype="bf16", Sq=50, H=21, H_k=3, S_max=400, seqlen=[400, 50], mask="causal"),
    "many_odd": dict(dtype="e4m3", Sq=333, H=20, H_k=2, S_max=1400, seqlen=[1400, 333, 700, 129], n_query=[333, 331, 40, 0],
                     mask="causal"),
    "many_no_mask": dict(dtype="f16", Sq=260, H=8, H_k=2, S_max=700, seqlen=[641, 0, 513], n_query=[260, 7, 259]),
    "batch": dict(dtype="bf16", Sq=2, H=8, H_k=2, S_max=500, seqlen=[(i * 41) % 501 for i in range(70)]),
}


@pytest.mark.parametrize("name", W_CASES)
def test_weights_match_the_formula(fm, name):
    c = make(seed=len(name), **W_CASES[name])
    was = torch.rand(c["acc"].shape, generator=torch.Generator().manual_seed(1))
    out = was.cuda()
    assert weights(fm, c, acc=c["acc"].cuda(), out=out) is out
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    check_weights(c, out, was)
    # in place gives the same bits below the lengths
    acc = c["acc"].cuda()
    assert weights(fm, c, acc=acc) is acc
    check_weights(c, acc, c["acc"])
    for e, L in zip(c["entry"], c["seqlen"]):
        assert torch.equal(acc[e, :, :L], out[e, :, :L])


# two chunks of queries: units that are left whole, or cut since they are more than the CTAs
W_TWO = {
    "whole": dict(dtype="bf16", Sq=40, H=16, H_k=4, S_max=700, seqlen=[700, 0, 40, 300], n_query=[40, 3, 0, 33], mask="causal"),
    "whole_e4m3": dict(dtype="e4m3", Sq=64, H=32, H_k=8, S_max=130, seqlen=[130, 64]),
    "whole_long": dict(dtype="f16", Sq=33, H=8, H_k=2, S_max=6000, seqlen=[6000, 33, 5119], mask="causal"),
    "whole_odd_group": dict(dtype="bf16", Sq=50, H=9, H_k=3, S_max=520, seqlen=[513, 50, 7, 512], n_query=[50, 50, 7, 43],
                            mask="causal"),
    "cut": dict(dtype="bf16", Sq=40, H=16, H_k=4, S_max=300, seqlen=[(i * 37) % 300 for i in range(60)],
                n_query=[min(40, (i * 37) % 300) for i in range(60)], mask="causal"),
}


@pytest.mark.parametrize("name", W_TWO)
def test_weights_of_two_chunks(fm, name):
    c = make(seed=70 + len(name), **W_TWO[name])
    out = torch.full(c["acc"].shape, 3.0, device="cuda")
    r = weights(fm, c, acc=c["acc"].cuda(), out=out)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    check_weights(c, r, torch.full(c["acc"].shape, 3.0))


def test_weights_from_nothing_and_of_rows_without_keys(fm):
    c = make("bf16", 4, 8, 2, 300, [290, 17], seed=4)
    c["want"] -= c["acc"].double()
    check_weights(c, weights(fm, c), torch.zeros_like(c["acc"]))
    # rows whose LSE says that they saw no key add nothing
    c["lse"][0] = -math.inf
    c["want"][0] = 0.0
    check_weights(c, weights(fm, c), torch.zeros_like(c["acc"]))


def test_weights_sum_to_the_number_of_rows(fm):
    """Every query row hands out a weight of 1 over the keys it sees."""
    c = make("bf16", 260, 8, 2, 1500, [1500, 777], mask="causal", seed=6)
    acc = weights(fm, c)
    for b, L in enumerate(c["seqlen"]):
        total = acc[b, :, :L].double().sum(-1).cpu()
        assert ((total - 260 * 4).abs() <= 260 * 4 * 1e-5).all()


def test_weights_report_bad_device_values(fm):
    c = make("bf16", 2, 4, 2, 100, [90, 50], n_query=[2, 1], batch_idx=[0, 1], seed=2)
    for key, bad in (("seqlen", [101, 50]), ("n_query", [3, 1]), ("batch_idx", [0, 7]), ("seqlen", [90, -1])):
        weights(fm, {**c, key: bad})
        assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG, (key, bad)
    got = weights(fm, {**c, "batch_idx": [0, 7]})
    assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG
    assert not got[1].any()                                   # nothing is written for a missing entry


def test_weights_in_graphs_on_two_streams(fm):
    cs = [make("bf16", 130, 8, 2, 900, [900, 500], mask="causal", seed=s) for s in (1, 2)]
    outs, graphs, streams, keep = [], [], [torch.cuda.Stream() for _ in cs], []
    for c in cs:
        out = torch.zeros(c["acc"].shape, device="cuda")
        args = [c["q"].cuda(), c["kc"].cuda(), c["lse"].cuda(), i32(c["seqlen"])]
        kw = dict(acc=c["acc"].cuda(), out=out, mask="causal",
                  workspace=torch.empty(fm.fmha_cache_weights_workspace_size(), dtype=torch.uint8, device="cuda"))
        fm.cache_weights(*args, **kw)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            fm.cache_weights(*args, **kw)
        outs.append((out, out.clone()))
        out.zero_()
        graphs.append(gr)
        keep.append((args, kw))
    torch.cuda.synchronize()
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for c, (out, eager) in zip(cs, outs):
        assert torch.equal(out, eager)
        check_weights(c, out, torch.zeros_like(c["acc"]))


# ---------------------------------------------------------------------------
# Eviction
# ---------------------------------------------------------------------------

def plain_kept(acc, L, budget, recent):
    """Rows that stay, ascending: the newest, and the largest scores (ties: lower row; NaN last)."""
    if L <= budget:
        return list(range(L))
    cand = acc[:L - recent].double()
    key = torch.where(torch.isnan(cand), torch.full_like(cand, -math.inf), cand).tolist()
    nan = torch.isnan(cand).tolist()
    best = sorted(range(L - recent), key=lambda j: (nan[j], -key[j], j))[:budget - recent]
    return sorted(best) + list(range(L - recent, L))


def scores(gen, shape, kind):
    if kind == "ties":
        return torch.randint(0, 4, shape, generator=gen).float()
    if kind == "equal":
        return torch.full(shape, 0.25)
    x = torch.randn(shape, generator=gen)
    if kind == "special":                                     # signed zeros, infinities, NaN, tiny numbers
        v = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 1e-45, -1e-45, 1e-38])
        return torch.where(torch.rand(shape, generator=gen) < 0.7, v[torch.randint(0, 8, shape, generator=gen)], x)
    return torch.exp(2 * x) * (torch.rand(shape, generator=gen) > 0.3)


E_CASES = {
    "heavy": dict(dtype="bf16", H_k=8, S_max=1500, S_out=600, seqlen=[1500, 601, 600, 599, 0, 1], budget=600, recent=64),
    "no_recent": dict(dtype="f16", H_k=3, S_max=700, S_out=129, seqlen=[700, 130], budget=129, recent=0),
    "only_recent": dict(dtype="bf16", H_k=2, S_max=300, S_out=40, seqlen=[300, 39], budget=40, recent=40),
    "budget_1": dict(dtype="e4m3", H_k=1, S_max=50, S_out=5, seqlen=[50, 2, 1], budget=1, recent=0),
    "all_but_one": dict(dtype="e4m3", H_k=5, S_max=1025, S_out=1024, seqlen=[1025], budget=1024, recent=3),
    "long": dict(dtype="e4m3", H_k=2, S_max=70001, S_out=1000, seqlen=[70001, 40000], budget=999, recent=10),
    "two_ctas": dict(dtype="bf16", H_k=3, S_max=4700, S_out=300, seqlen=[4700, 301], budget=300, recent=7),
    "many": dict(dtype="bf16", H_k=2, S_max=90, S_out=64, seqlen=[(i * 17) % 91 for i in range(80)], budget=33, recent=5),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "special"])
@pytest.mark.parametrize("name", E_CASES)
def test_evict_keeps_and_moves_what_it_says(fm, name, kind, in_place):
    a = E_CASES[name]
    if a["S_max"] > 10000 and (kind == "equal" or in_place and kind != "ties"):
        pytest.skip("the long case runs with three kinds of scores")
    g = torch.Generator().manual_seed(len(name))
    B, H_k, S, budget, recent = len(a["seqlen"]), a["H_k"], a["S_max"], a["budget"], a["recent"]
    bidx = torch.randperm(B, generator=g).tolist()
    oidx = bidx if in_place else torch.randperm(B, generator=g).tolist()
    k, v = (cu.draw(g, (B, S, H_k, 128), a["dtype"]) for _ in range(2))
    acc = scores(g, (B, H_k, S), kind)
    kd, vd, ad = k.cuda(), v.cuda(), acc.cuda()
    bi = i32(bidx)
    if in_place:
        ko, vo, ao, kw = kd, vd, ad, {}
        k0, v0, S_out = k.clone(), v.clone(), S
    else:
        S_out = a["S_out"]
        ko, vo = (cu.sentinel((B, S_out, H_k, 128), cu.DTYPES[a["dtype"]]) for _ in range(2))
        ao = cu.sentinel((B, H_k, S_out), torch.float32)
        k0, v0 = ko.cpu(), vo.cpu()
        kw = dict(k_out=ko, v_out=vo, acc_out=ao, out_idx=i32(oidx))
    kept, new = fm.cache_evict(kd, vd, ad, i32(a["seqlen"]), budget, recent=recent, batch_idx=bi, **kw)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    want_acc = torch.zeros((B, H_k, S_out))
    for b, L in enumerate(a["seqlen"]):
        n = min(L, budget)
        assert int(new[b]) == n
        for h in range(H_k):
            rows = plain_kept(acc[bidx[b], h], L, budget, recent)
            assert kept[b, h].tolist() == rows + [-1] * (budget - n), (b, h)
            k0[oidx[b], :n, h], v0[oidx[b], :n, h] = cu.take(k[bidx[b], :, h], rows), cu.take(v[bidx[b], :, h], rows)
            want_acc[oidx[b], h, :n] = acc[bidx[b], h, rows]
    assert torch.equal(ko.cpu().view(torch.uint8), k0.view(torch.uint8))
    assert torch.equal(vo.cpu().view(torch.uint8), v0.view(torch.uint8))
    assert torch.equal(ao.cpu().view(torch.int32), want_acc.view(torch.int32))


def test_evict_reports_bad_device_values_and_moves_nothing_for_them(fm):
    g = torch.Generator().manual_seed(1)
    k, v = (cu.draw(g, (2, 40, 2, 128), "bf16").cuda() for _ in range(2))
    acc = torch.rand((2, 2, 40), generator=g).cuda()
    for key, bad in (("batch_idx", [0, 2]), ("out_idx", [-1, 1]), ("seqlen", [41, 10]), ("seqlen", [40, -1])):
        ko, vo = (cu.sentinel((2, 8, 2, 128), torch.bfloat16) for _ in range(2))
        ao = cu.sentinel((2, 2, 8), torch.float32)
        a = {"batch_idx": [0, 1], "out_idx": [0, 1], "seqlen": [40, 10], key: bad}
        fm.cache_evict(k, v, acc, i32(a["seqlen"]), 8, recent=2, batch_idx=i32(a["batch_idx"]), k_out=ko, v_out=vo,
                       acc_out=ao, out_idx=i32(a["out_idx"]))
        assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG, (key, bad)
        if key != "seqlen":
            b = 0 if key == "out_idx" else 1
            assert cu.untouched(ko[b]) and cu.untouched(vo[b]) and cu.untouched(ao[b])


def test_evict_replays_in_a_graph(fm):
    g = torch.Generator().manual_seed(9)
    k, v = (cu.draw(g, (2, 500, 2, 128), "bf16").cuda() for _ in range(2))
    acc, sl = torch.rand((2, 2, 500), generator=g).cuda(), i32([500, 450])
    out = lambda: dict(k_out=torch.zeros((2, 100, 2, 128), dtype=torch.bfloat16, device="cuda"),
                       v_out=torch.zeros((2, 100, 2, 128), dtype=torch.bfloat16, device="cuda"),
                       acc_out=torch.zeros((2, 2, 100), device="cuda"), kept=torch.zeros((2, 2, 100), dtype=torch.int32, device="cuda"),
                       new_seqlen=torch.zeros((2,), dtype=torch.int32, device="cuda"))
    a, b = out(), out()
    fm.cache_evict(k, v, acc, sl, 100, recent=10, **a)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        fm.cache_evict(k, v, acc, sl, 100, recent=10, **b)
    acc.copy_(torch.rand((2, 2, 500), generator=g))           # other scores: the replay selects by them
    gr.replay()
    fm.cache_evict(k, v, acc, sl, 100, recent=10, **a)
    torch.cuda.synchronize()
    for key in a:
        assert torch.equal(a[key], b[key]), key


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_decode_loop_with_drafts_and_eviction(fm, dtype):
    """Generation steps and verified drafts fill a cache, their weights are
    accumulated, and it is shrunk in place when it is nearly full.  Beside it a
    plain cache (tensors per sequence and head, in 64 bits where numbers are
    computed) takes the same steps on the same stored values."""
    g = torch.Generator().manual_seed(11)
    B, H, H_k, S, T, budget, recent = 3, 8, 2, 260, 6, 96, 16
    G = H // H_k
    L = [200, 255, 7]
    kc, vc = (cu.draw(g, (B, S, H_k, 128), dtype).cuda() for _ in range(2))
    acc = torch.zeros((B, H_k, S), device="cuda")
    entry = [2, 0, 1]
    bidx, sl = i32(entry), i32(L)
    mirror = [[dict(k=kc[e, :n, h].cpu(), v=vc[e, :n, h].cpu(), a=torch.zeros(n).double()) for h in range(H_k)]
              for e, n in zip(entry, L)]
    for step in range(12):
        if max(L) + T > S:
            kept, new = fm.cache_evict(kc, vc, acc, sl, budget, recent=recent, batch_idx=bidx)
            for b in range(B):
                n = min(L[b], budget)
                for h in range(H_k):
                    # the loop's own fp32 scores choose; the move is checked against them
                    m, rows = mirror[b][h], kept[b, h, :n].long().cpu()
                    mirror[b][h] = dict(k=cu.take(m["k"], rows), v=cu.take(m["v"], rows), a=m["a"][rows])
                L[b] = n
            sl = new
            assert sl.tolist() == L
        tree = step % 3 == 2
        t = T if tree else 1
        q = cu.draw(g, (B, t, H, 128), dtype, 2.0)
        kn, vn = (cu.draw(g, (B, t, H_k, 128), dtype) for _ in range(2))
        mask = cu.random_tree(g, B, t)
        if tree:
            o, lse = fm.tree_fwd(q.cuda(), kc, vc, kn.cuda(), vn.cuda(), sl, tree_mask=mask.cuda(), batch_idx=bidx)
        else:
            o, lse = fm.gen_fwd(q[:, 0].contiguous().cuda(), kc, vc, sl, k_new=kn[:, 0].contiguous().cuda(),
                                v_new=vn[:, 0].contiguous().cuda(), batch_idx=bidx)
            o, lse = o.unsqueeze(1), lse.unsqueeze(-1)
        fm.cache_weights(q.cuda(), kc, lse.contiguous(), sl, acc=acc, batch_idx=bidx)
        path, n_acc = [], []
        for b in range(B):
            n_acc.append(int(torch.randint(1, t + 1, (1,), generator=g)) if tree else 1)
            path.append(torch.randperm(t, generator=g)[:n_acc[-1]].sort().values.tolist() + [0] * (t - n_acc[-1]))
        if tree:
            fm.tree_commit(kc, vc, kn.cuda(), vn.cuda(), sl, i32(path), i32(n_acc), batch_idx=bidx)
        for b in range(B):
            see = torch.cat([torch.ones((t, L[b]), dtype=torch.bool), mask[b]], 1)
            for h in range(H_k):
                m = mirror[b][h]
                keys, vals = torch.cat([m["k"], kn[b, :, h]]), torch.cat([m["v"], vn[b, :, h]])
                qh = cu.f64(q[b, :, h * G:(h + 1) * G])
                want, wl, tol, tl = cu.attend(qh, cu.f64(keys), cu.f64(vals), see, 128 ** -0.5, 1.0, dtype)
                cu.close(cu.f64(o[b, :, h * G:(h + 1) * G].cpu()), want, tol, f"O at step {step}")
                cu.close(lse[b, h * G:(h + 1) * G].double().cpu().T, wl, tl, f"LSE at step {step}")
                w = torch.exp(torch.einsum("tgd,kd->tgk", qh, cu.f64(m["k"])) * 128 ** -0.5 - wl[..., None])
                rows = path[b][:n_acc[b]]
                mirror[b][h] = dict(k=torch.cat([m["k"], cu.take(kn[b, :, h], rows)]),
                                    v=torch.cat([m["v"], cu.take(vn[b, :, h], rows)]),
                                    a=torch.cat([m["a"] + w.sum((0, 1)), torch.zeros(len(rows)).double()]))
            L[b] += n_acc[b]
        sl = sl + i32(n_acc)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    for b in range(B):
        for h in range(H_k):
            m = mirror[b][h]
            assert torch.equal(kc[entry[b], :L[b], h].cpu().view(torch.uint8), m["k"].view(torch.uint8))
            assert torch.equal(vc[entry[b], :L[b], h].cpu().view(torch.uint8), m["v"].view(torch.uint8))
            # 12 steps of at most T * G weights, each off by a few 2^-23 of its score's terms (30 at most here)
            assert ((acc[entry[b], h, :L[b]].double().cpu() - m["a"]).abs() <= m["a"] * 130 * 30 * 2.0 ** -23 * 2 + 1e-6).all()
