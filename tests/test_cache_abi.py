"""Argument checks of the cache operators' entry points, without a GPU: every
refusal comes before the device is looked at."""
import pytest
import torch

P, P2, P3 = 0x10000000, 0x20000000, 0x30000000       # fake, aligned, far apart: never dereferenced
F16, BF16, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def fm():
    from head_attention_forward_02_gb300 import build, fmha
    build.build()
    fmha.lib()
    return fmha


def tensors(fm, a, names, dt):
    return [fm.fmha_tensor(a[n], a.get(n + "_dt", dt)) for n in names]


def call_tree(fm, **kw):
    a = dict(q=P, kc=P, vc=P, kn=P, vn=P, o=P, lse=None, B=2, T=4, H=8, H_k=2, D=128, Bc=2, S=64, sl=P, bi=None, nd=None,
             mask=None, ms=0, scale=0.1, out_scale=1.0, ws=P, ws_bytes=1 << 30, dt=BF16)
    a.update(kw)
    t = tensors(fm, a, ("q", "kc", "vc", "kn", "vn", "o"), a["dt"])
    return fm.lib().fmha_tree_fwd(*t, a["lse"], a["B"], a["T"], a["H"], a["H_k"], a["D"], a["Bc"], a["S"], a["sl"],
                                  a["bi"], a["nd"], a["mask"], a["ms"], a["scale"], a["out_scale"], a["ws"],
                                  a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), -1), (dict(H=3), -1), (dict(H=129, H_k=1), -1), (dict(H_k=0), -1), (dict(B=-1), -1), (dict(T=-1), -1),
    (dict(S=0), -1), (dict(Bc=0), -1), (dict(sl=None), -1), (dict(scale=0.0), -1), (dict(scale=float("inf")), -1),
    (dict(scale=float("nan")), -1), (dict(out_scale=float("nan")), -1), (dict(out_scale=float("inf")), -1),
    (dict(mask=P, ms=15), -1), (dict(mask=P, ms=-16), -1), (dict(ws=None), -1), (dict(ws=P + 128), -1),
    (dict(ws_bytes=1000), -1), (dict(lse=P + 2), -1), (dict(sl=P + 2), -1), (dict(nd=P + 1), -1), (dict(bi=P + 3), -1),
    *[({n: None}, -1) for n in ("q", "kc", "vc", "kn", "vn", "o")],
    *[({n: P + 8}, -2) for n in ("q", "kc", "vc", "kn", "vn", "o")],
    *[({n + "_dt": F16}, -2) for n in ("kc", "vc", "kn", "vn", "o")],
    (dict(dt=5), -2), (dict(B=1 << 20, T=1 << 10), -1), (dict(S=(1 << 30) + 1), -1),
    (dict(B=0, q=None, sl=None, ws=None), 0), (dict(T=0, q=None, sl=None, ws=None), 0),
])
def test_tree_refusals(fm, kw, code):
    assert call_tree(fm, **kw) == code


def test_tree_workspace_size(fm):
    size = fm.fmha_tree_workspace_size
    row = 128 * (128 + 1) * 4                               # a 128-row block: fp32 O and LSE
    meta = 20
    # one block of rows: B * H_k * (key tiles + draft tiles) tiles, a CTA each up to 152, two slots a CTA
    assert size(1, 8, 32, 8, 128, 1000) == 2 * 8 * 9 * (row + meta)
    assert size(64, 8, 32, 8, 128, 100000) == 2 * 152 * (row + meta)
    # more rows than a block holds: two a unit
    assert size(64, 33, 32, 8, 128, 100000) == 2 * 152 * (2 * row + meta)
    assert size(64, 33, 32, 8, 128, 100000) <= 41 << 20
    for bad in [(0, 8, 32, 8, 128, 10), (1, 0, 32, 8, 128, 10), (1, 8, 3, 2, 128, 10), (1, 8, 32, 8, 64, 10),
                (1, 8, 32, 8, 128, 0), (1, 8, 129, 1, 128, 10),
                (1, 8, 32, 8, 128, (1 << 30) + 1)]:
        assert size(*bad) == 0


def call_commit(fm, **kw):
    a = dict(kc=P, vc=P, kn=P, vn=P, B=2, T=4, P=3, H_k=2, D=128, Bc=2, S=64, sl=P, bi=None, path=P, na=P, dt=BF16)
    a.update(kw)
    t = tensors(fm, a, ("kc", "vc", "kn", "vn"), a["dt"])
    return fm.lib().fmha_tree_commit(*t, a["B"], a["T"], a["P"], a["H_k"], a["D"], a["Bc"], a["S"], a["sl"], a["bi"],
                                     a["path"], a["na"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), -1), (dict(H_k=0), -1), (dict(B=-1), -1), (dict(P=-1), -1), (dict(T=0), -1), (dict(S=0), -1),
    (dict(Bc=0), -1), (dict(sl=None), -1), (dict(path=None), -1), (dict(na=None), -1), (dict(path=P + 2), -1),
    *[({n: None}, -1) for n in ("kc", "vc", "kn", "vn")], *[({n: P + 8}, -2) for n in ("kc", "vc", "kn", "vn")],
    (dict(vn_dt=F16), -2), (dict(dt=9), -2), (dict(B=70000), -2), (dict(S=(1 << 30) + 1), -1),
    (dict(B=0, kc=None, sl=None), 0), (dict(P=0, path=None, sl=None), 0),
])
def test_commit_refusals(fm, kw, code):
    assert call_commit(fm, **kw) == code


def call_weights(fm, **kw):
    a = dict(q=P, kc=P, lse=P, ai=P2, ao=P3, B=2, Sq=4, H=8, H_k=2, D=128, Bc=2, S=64, sl=P, bi=None, nq=None, scale=0.1,
             mask=0, ws=P, ws_bytes=1 << 30, dt=BF16)
    a.update(kw)
    t = tensors(fm, a, ("q", "kc"), a["dt"])
    return fm.lib().fmha_cache_weights(*t, a["lse"], a["ai"], a["ao"], a["B"], a["Sq"], a["H"], a["H_k"], a["D"], a["Bc"],
                                       a["S"], a["sl"], a["bi"], a["nq"], a["scale"], a["mask"], a["ws"],
                                       a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=32), -1), (dict(H=3), -1), (dict(H=129, H_k=1), -1), (dict(B=-1), -1), (dict(Sq=-1), -1), (dict(S=0), -1),
    (dict(Bc=0), -1), (dict(sl=None), -1), (dict(lse=None), -1), (dict(ao=None), -1), (dict(q=None), -1),
    (dict(kc=None), -1), (dict(scale=-1.0), -1), (dict(mask=1), -1), (dict(mask=3), -1), (dict(ws=None), -1),
    (dict(ws=P + 16), -1), (dict(ws_bytes=16), -1), (dict(lse=P + 2), -1), (dict(ai=P2 + 1), -1),
    (dict(ao=P2 + 4), -1), (dict(ai=P3 + 4 * 2 * 2 * 64 - 4), -1),      # neither the same array nor apart
    (dict(q=P + 8), -2), (dict(kc=P + 8), -2), (dict(kc_dt=E4M3), -2), (dict(dt=4), -2), (dict(S=(1 << 30) + 1), -1),
    (dict(B=0, q=None, ws=None), 0), (dict(Sq=0, q=None, ws=None), 0),
])
def test_weights_refusals(fm, kw, code):
    assert call_weights(fm, **kw) == code


def call_evict(fm, **kw):
    a = dict(kc=P, vc=2 * P, acc=3 * P, ko=4 * P, vo=5 * P, ao=6 * P, B=2, H_k=2, D=128, Bc=2, S=64, Bo=2, So=40, sl=P,
             bi=None, oi=None, budget=32, recent=4, kept=P, ns=P2, dt=BF16)
    a.update(kw)
    k = tensors(fm, a, ("kc", "vc", "ko", "vo"), a["dt"])
    return fm.lib().fmha_cache_evict(k[0], k[1], a["acc"], k[2], k[3], a["ao"], a["B"], a["H_k"], a["D"], a["Bc"], a["S"],
                                     a["Bo"], a["So"], a["sl"], a["bi"], a["oi"], a["budget"], a["recent"], a["kept"],
                                     a["ns"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), -1), (dict(H_k=0), -1), (dict(B=-1), -1), (dict(budget=0), -1), (dict(budget=41), -1),
    (dict(recent=-1), -1), (dict(recent=33), -1), (dict(S=0), -1), (dict(So=0), -1), (dict(Bc=0), -1), (dict(Bo=0), -1),
    (dict(sl=None), -1), (dict(kept=None), -1), (dict(ns=None), -1), (dict(ns=P), -1), (dict(acc=None), -1),
    (dict(ao=None), -1), (dict(ao=6 * P + 2), -1),
    *[({n: None}, -1) for n in ("kc", "vc", "ko", "vo")], *[({n: 7 * P + 8}, -2) for n in ("kc", "vc", "ko", "vo")],
    (dict(vo_dt=E4M3), -2), (dict(dt=3), -2), (dict(B=70000), -2), (dict(S=(1 << 30) + 1), -1),
    (dict(So=(1 << 30) + 1), -1),
    # in place means all three arrays, with the sizes and entries of the input
    (dict(ko=P), -1), (dict(ko=P, vo=2 * P, ao=3 * P), -1), (dict(ko=P, vo=2 * P, ao=3 * P, So=64, oi=P3), -1),
    # else the output is apart from the input
    (dict(ko=P + 16), -1), (dict(vo=P), -1), (dict(ao=3 * P), -1), (dict(ko=3 * P), -1),
    (dict(B=0, kc=None, sl=None), 0),
])
def test_evict_refusals(fm, kw, code):
    assert call_evict(fm, **kw) == code


def test_outputs_over_inputs_are_refused(fm):
    a = dict(q=P, kc=2 * P, vc=3 * P, kn=4 * P, vn=5 * P, ws=6 * P)
    for n in ("q", "kc", "vc", "kn", "vn"):
        size = 2 * 128 * 2 * (64 * 2 if n in ("kc", "vc") else 4 * (8 if n == "q" else 2))       # bytes
        assert call_tree(fm, **a, o=a[n]) == -1
        assert call_tree(fm, **a, o=a[n] + size - 16) == -1
    c = dict(kc=P, vc=2 * P, kn=3 * P, vn=4 * P)
    for x, y in (("kc", "vc"), ("kc", "kn"), ("kc", "vn"), ("vc", "kn"), ("vc", "vn")):
        assert call_commit(fm, **{**c, y: c[x]}) == -1
        assert call_commit(fm, **{**c, y: c[x] + 2 * 64 * 2 * 128 * 2 - 16}) == -1               # the cache's last bytes


def test_host_tensors_are_refused(fm):
    q = torch.zeros((1, 2, 4, 128), dtype=torch.bfloat16)
    i = torch.zeros((1,), dtype=torch.int32)
    f = torch.zeros((1, 4, 2))
    for call in (lambda: fm.tree_fwd(q, q, q, q, q, i), lambda: fm.tree_commit(q, q, q, q, i, i[None], i),
                 lambda: fm.cache_weights(q, q, f, i), lambda: fm.cache_evict(q, q, f, i, 1)):
        with pytest.raises(ValueError):
            call()
