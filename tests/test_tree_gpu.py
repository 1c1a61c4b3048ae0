"""Attention of drafted trees over a K/V cache (fmha_tree_fwd) and the commit
of accepted drafts, on the GPU, against their formulas in 64 bits."""
import pytest
import torch

from tests import cache_util as cu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_attention_forward_02_gb300 import build, fmha
    build.build()
    fmha.lib()
    return fmha


def make(dtype, T, H, H_k, S_max, seqlen, n_draft=None, mask="tree", batch_idx=None, seed=0, q_scale=2.0):
    g = torch.Generator().manual_seed(seed)
    B = len(seqlen)
    B_cache = B if batch_idx is None else max(batch_idx) + 1
    c = dict(dtype=dtype, B=B, T=T, H=H, H_k=H_k, seqlen=list(seqlen), n=list(n_draft) if n_draft else [T] * B,
             entry=list(batch_idx) if batch_idx else list(range(B)), has_n=n_draft is not None,
             has_idx=batch_idx is not None)
    c["q"] = cu.draw(g, (B, T, H, 128), dtype, q_scale)
    c["kc"], c["vc"] = (cu.draw(g, (B_cache, S_max, H_k, 128), dtype) for _ in range(2))
    c["kn"], c["vn"] = (cu.draw(g, (B, T, H_k, 128), dtype) for _ in range(2))
    if mask == "chain":
        c["mask"] = None
    elif mask == "shared":
        c["mask"] = cu.random_tree(g, 1, T)[0]
    elif mask == "any":                        # not a tree: rows that see nothing of the drafts among them
        c["mask"] = torch.rand((B, T, T), generator=g) < 0.4
        c["mask"][:, ::3] = False
    else:
        c["mask"] = cu.random_tree(g, B, T)
    last = {}
    for e, L in zip(c["entry"], c["seqlen"]):
        last[e] = max(last.get(e, 0), L)
    for e in range(B_cache):                   # rows past every length hold NaN
        cu.fill_nan(c["kc"], (e, slice(last.get(e, 0), None)))
        cu.fill_nan(c["vc"], (e, slice(last.get(e, 0), None)))
    for b, n in enumerate(c["n"]):
        for t in ("q", "kn", "vn"):
            cu.fill_nan(c[t], (b, slice(n, None)))
    return c


def on_gpu(c):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    return dict(args=[c[t].cuda() for t in ("q", "kc", "vc", "kn", "vn")] + [i32(c["seqlen"])],
                kw=dict(tree_mask=None if c["mask"] is None else c["mask"].cuda(),
                        n_draft=i32(c["n"]) if c["has_n"] else None,
                        batch_idx=i32(c["entry"]) if c["has_idx"] else None))


def outputs(c):
    dt = cu.DTYPES[c["dtype"]]
    return cu.sentinel((c["B"], c["T"], c["H"], 128), dt), cu.sentinel((c["B"], c["H"], c["T"]), torch.float32)


def check(c, o, lse, scale=128 ** -0.5, out_scale=1.0):
    o, lse = o.cpu(), lse.cpu()
    G = c["H"] // c["H_k"]
    for b in range(c["B"]):
        L, n, e = c["seqlen"][b], c["n"][b], c["entry"][b]
        assert cu.untouched(o[b, n:]) and cu.untouched(lse[b, :, n:]), f"rows past the drafts of sequence {b}"
        tree = torch.ones((n, n), dtype=torch.bool).tril() if c["mask"] is None else \
            (c["mask"] if c["mask"].dim() == 2 else c["mask"][b])[:n, :n]
        see = torch.cat([torch.ones((n, L), dtype=torch.bool), tree], 1)
        for g in range(c["H_k"]):
            keys = torch.cat([cu.f64(c["kc"][e, :L, g]), cu.f64(c["kn"][b, :n, g])])
            vals = torch.cat([cu.f64(c["vc"][e, :L, g]), cu.f64(c["vn"][b, :n, g])])
            q = cu.f64(c["q"][b, :n, g * G:(g + 1) * G])
            want, wl, tol, tl = cu.attend(q, keys, vals, see, scale, out_scale, c["dtype"])
            cu.close(cu.f64(o[b, :n, g * G:(g + 1) * G]), want, tol, f"O of sequence {b} head {g}")
            cu.close(lse[b, g * G:(g + 1) * G, :n].double().T, wl, tl, f"LSE of sequence {b} head {g}")


CASES = {
    "one_token_empty_cache": dict(dtype="bf16", T=1, H=8, H_k=8, S_max=16, seqlen=[0], mask="chain"),
    "one_token_one_key": dict(dtype="f16", T=1, H=4, H_k=1, S_max=1, seqlen=[1], mask="chain"),
    "latency": dict(dtype="bf16", T=8, H=32, H_k=8, S_max=1000, seqlen=[1000]),
    "split_many": dict(dtype="bf16", T=5, H=4, H_k=1, S_max=20000, seqlen=[19999]),
    "odd_group": dict(dtype="bf16", T=7, H=9, H_k=3, S_max=300, seqlen=[127, 128, 129, 0], n_draft=[7, 1, 3, 5]),
    "group_of_128": dict(dtype="f16", T=3, H=128, H_k=1, S_max=260, seqlen=[257, 13]),
    "group_of_65": dict(dtype="bf16", T=3, H=65, H_k=1, S_max=130, seqlen=[130]),
    "two_blocks": dict(dtype="bf16", T=64, H=8, H_k=2, S_max=700, seqlen=[641, 0, 512], n_draft=[64, 33, 32]),
    "three_blocks": dict(dtype="f16", T=40, H=16, H_k=2, S_max=400, seqlen=[300, 399], n_draft=[40, 17]),
    "two_draft_tiles": dict(dtype="bf16", T=131, H=2, H_k=2, S_max=200, seqlen=[77, 200, 0], n_draft=[131, 128, 129]),
    "wide_draft_group": dict(dtype="e4m3", T=70, H=20, H_k=4, S_max=500, seqlen=[499, 128], n_draft=[70, 69]),
    "shared_mask": dict(dtype="bf16", T=13, H=8, H_k=2, S_max=140, seqlen=[3, 140], mask="shared"),
    "rows_without_keys": dict(dtype="bf16", T=20, H=8, H_k=2, S_max=64, seqlen=[0, 0, 5], n_draft=[20, 9, 20], mask="any"),
    "no_drafts": dict(dtype="bf16", T=4, H=8, H_k=2, S_max=300, seqlen=[300, 200, 0], n_draft=[0, 4, 0]),
    "shared_entry": dict(dtype="f16", T=6, H=8, H_k=4, S_max=500, seqlen=[400, 400, 17], batch_idx=[2, 2, 0]),
    "e4m3_small": dict(dtype="e4m3", T=4, H=16, H_k=2, S_max=1100, seqlen=[1100, 700], batch_idx=[1, 0]),
    "batch": dict(dtype="bf16", T=9, H=8, H_k=2, S_max=900, seqlen=[(i * 37) % 900 for i in range(70)],
                  n_draft=[1 + i % 9 for i in range(70)], batch_idx=[(i * 3) % 70 for i in range(70)]),
    "peaked": dict(dtype="bf16", T=12, H=8, H_k=2, S_max=3000, seqlen=[2999], q_scale=20.0),
    "head_pairs": dict(dtype="e4m3", T=3, H=40, H_k=10, S_max=4500, seqlen=[4500, 130, 0, 4097, 128, 700], n_draft=[3, 1, 3, 0, 2, 3],
                       batch_idx=[5, 0, 2, 1, 4, 3]),
    "head_pairs_full": dict(dtype="e4m3", T=32, H=16, H_k=4, S_max=9000, seqlen=[9000, 20, 4097, 128, 333]),
    "wide_long": dict(dtype="e4m3", T=64, H=8, H_k=1, S_max=4100, seqlen=[4097]),
}


@pytest.mark.parametrize("name", CASES)
def test_tree_matches_the_formula(fm, name):
    c = make(seed=len(name), **CASES[name])
    d, (o, lse) = on_gpu(c), outputs(c)
    fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    check(c, o, lse)


# the same lengths in caches whose size leaves units whole, or has them cut
SIZES = {
    "one_block": dict(dtype="bf16", T=7, H=9, H_k=3, seqlen=[127, 128, 129, 0, 300], n_draft=[7, 1, 3, 5, 0]),
    "two_blocks": dict(dtype="f16", T=64, H=8, H_k=2, seqlen=[541, 0, 512, 130], n_draft=[64, 33, 32, 1]),
    "three_blocks": dict(dtype="e4m3", T=40, H=16, H_k=2, seqlen=[300, 399], n_draft=[40, 17]),
    "two_draft_tiles": dict(dtype="bf16", T=131, H=2, H_k=2, seqlen=[77, 200, 0], n_draft=[131, 128, 129]),
    "rows_without_keys": dict(dtype="bf16", T=20, H=8, H_k=2, seqlen=[0, 0, 5], n_draft=[20, 9, 20], mask="any"),
    "more_units_than_ctas": dict(dtype="bf16", T=3, H=8, H_k=8, seqlen=[(i * 41) % 250 for i in range(50)],
                                 n_draft=[i % 4 for i in range(50)]),
}


@pytest.mark.parametrize("S_max", [600, 5000])
@pytest.mark.parametrize("name", SIZES)
def test_tree_of_whole_and_of_cut_units(fm, name, S_max):
    c = make(seed=50 + len(name), S_max=S_max, **SIZES[name])
    d, (o, lse) = on_gpu(c), outputs(c)
    fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    check(c, o, lse)


def test_tree_scales_and_no_lse(fm):
    c = make("bf16", 6, 8, 2, 300, [290, 3], seed=5)
    d, (o, lse) = on_gpu(c), outputs(c)
    fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse, scale=0.03, out_scale=-1.5)
    check(c, o, lse, scale=0.03, out_scale=-1.5)
    o2, none = fm.tree_fwd(*d["args"], **d["kw"], scale=0.03, out_scale=-1.5, return_lse=False)
    assert none is None and torch.equal(o2, o)


def test_tree_of_one_token_agrees_with_generation(fm):
    """T = 1 is a generation step: the same keys, so the same LSE within the two bounds."""
    c = make("bf16", 1, 32, 8, 1500, [1499, 700, 0], mask="chain", seed=8)
    d, (o, lse) = on_gpu(c), outputs(c)
    fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse)
    check(c, o, lse)
    q, kc, vc, kn, vn, sl = d["args"]
    _, lg = fm.gen_fwd(q[:, 0].contiguous(), kc, vc, sl, k_new=kn[:, 0].contiguous(), v_new=vn[:, 0].contiguous())
    assert (lg - lse[:, :, 0]).abs().max().item() <= 2e-3


def test_tree_repeats_bit_for_bit_and_in_graphs_on_two_streams(fm):
    """Two captured calls with workspaces of their own, replayed at the same time, and the eager call agree bit for bit."""
    cs = [make("bf16", 33, 16, 4, 2000, [1999, 513, 64], n_draft=[33, 20, 1], seed=s) for s in (1, 2)]
    ds = [on_gpu(c) for c in cs]
    eager = [fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=l) for c, d in zip(cs, ds) for o, l in [outputs(c)]]
    torch.cuda.synchronize()
    outs = [outputs(c) for c in cs]
    ws = [torch.empty(fm.fmha_tree_workspace_size(3, 33, 16, 4, 128, 2000), dtype=torch.uint8, device="cuda") for _ in cs]
    graphs, streams = [], [torch.cuda.Stream() for _ in cs]
    for d, (o, l), w in zip(ds, outs, ws):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=l, workspace=w)
        graphs.append(gr)
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for (o, l), (oe, le), c in zip(outs, eager, cs):
        assert torch.equal(o.view(torch.int16), oe.view(torch.int16))
        assert torch.equal(l.view(torch.int32), le.view(torch.int32))
        check(c, o, l)


def test_tree_reports_bad_device_values(fm):
    c = make("bf16", 4, 8, 2, 200, [100, 50], n_draft=[4, 4], batch_idx=[0, 1], seed=3)
    for key, bad in (("n_draft", [4, 5]), ("n_draft", [-1, 4]), ("batch_idx", [0, 2]), ("batch_idx", [-1, 1]),
                     ("seqlen", [201, 50]), ("seqlen", [100, -7])):
        d, (o, lse) = on_gpu(c), outputs(c)
        v = torch.tensor(bad, dtype=torch.int32, device="cuda")
        if key == "seqlen":
            d["args"][5] = v
        else:
            d["kw"][key] = v
        fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse)
        assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG, (key, bad)
        fm.tree_fwd(*on_gpu(c)["args"], **on_gpu(c)["kw"], out=o, lse=lse)
        assert fm.device_status(reset=True) == 0
        check(c, o, lse)


# ---------------------------------------------------------------------------
# Commit
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,H_k,T,path,n_accept,seqlen,entry", [
    ("bf16", 8, 8, [[0, 2, 5, 7, -1]], [4], [3], None),
    ("e4m3", 1, 3, [[2, 2], [0, -9], [1, 0]], [2, 0, 2], [0, 30, 28], [1, 2, 0]),
    ("f16", 3, 70, [list(range(69, 2, -1)), list(range(67))], [67, 1], [500, 0], [1, 0]),
    ("bf16", 40, 2, [[1]], [1], [29], None),
])
def test_commit_moves_the_accepted_rows_only(fm, dtype, H_k, T, path, n_accept, seqlen, entry):
    g = torch.Generator().manual_seed(T)
    B, S = len(path), max(L + n for L, n in zip(seqlen, n_accept))
    kc, vc = (cu.draw(g, (B, S, H_k, 128), dtype) for _ in range(2))
    kn, vn = (cu.draw(g, (B, T, H_k, 128), dtype) for _ in range(2))
    i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")
    kd, vd = kc.cuda(), vc.cuda()
    fm.tree_commit(kd, vd, kn.cuda(), vn.cuda(), i32(seqlen), i32(path), i32(n_accept), batch_idx=i32(entry))
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    for b in range(B):
        for i in range(n_accept[b]):
            kc[entry[b] if entry else b, seqlen[b] + i] = kn[b, path[b][i]]
            vc[entry[b] if entry else b, seqlen[b] + i] = vn[b, path[b][i]]
    assert torch.equal(kd.cpu().view(torch.uint8), kc.view(torch.uint8))
    assert torch.equal(vd.cpu().view(torch.uint8), vc.view(torch.uint8))


def test_commit_reports_bad_device_values_and_writes_nothing_for_them(fm):
    g = torch.Generator().manual_seed(1)
    kc, vc = (cu.draw(g, (2, 10, 2, 128), "bf16").cuda() for _ in range(2))
    kn, vn = (cu.draw(g, (2, 4, 2, 128), "bf16").cuda() for _ in range(2))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    good = dict(seqlen=[3, 5], path=[[0, 1], [2, 3]], n_accept=[0, 2], batch_idx=[0, 1])
    for key, bad in (("path", [[0, 1], [4, -1]]), ("batch_idx", [0, 2]), ("seqlen", [3, 10]), ("n_accept", [0, -1])):
        a = {k: i32(v) for k, v in {**good, key: bad}.items()}
        k, v = kc.clone(), vc.clone()
        fm.tree_commit(k, v, kn, vn, a["seqlen"], a["path"], a["n_accept"], batch_idx=a["batch_idx"])
        assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG, (key, bad)
        assert torch.equal(k, kc) and torch.equal(v, vc), (key, bad)
    # a count past the cache's end is cut there
    k, v = kc.clone(), vc.clone()
    fm.tree_commit(k, v, kn, vn, i32([3, 9]), i32(good["path"]), i32([0, 2]))
    assert fm.device_status(reset=True) == fm.ERR_INVALID_ARG
    assert torch.equal(k[1, 9], kn[1, 2]) and torch.equal(k[:, :9], kc[:, :9])
