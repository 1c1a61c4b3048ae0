"""Argument checks of the paged-cache operators' entry points, without a GPU:
every refusal comes before the device is looked at."""
import pytest
import torch

F16, BF16, E4M3 = 0, 1, 2
M = 1 << 32                                              # fake addresses, far apart: never dereferenced


def apart(*names):
    return {n: (i + 1) * M for i, n in enumerate(names)}


@pytest.fixture(scope="module")
def fm():
    from head_attention_forward_02_gb300 import build, fmha
    build.build()
    fmha.lib()
    return fmha


@pytest.fixture
def no_device():
    if torch.cuda.is_available():
        pytest.skip("a device would be given the fake addresses")


# ---------------------------------------------------------------------------
# Plan: 3 sequences, 10 rows, a table of 4 rows of 8, 20 pages of 16
# ---------------------------------------------------------------------------

PLAN = apart("sl", "nn", "bi", "tab", "free", "nf", "nfo", "slots", "pos", "cu", "ns")
PLAN_BYTES = dict(sl=12, nn=12, bi=12, tab=4 * 8 * 4, free=80, nf=4, nfo=4, slots=40, pos=40, cu=16, ns=12)


def call_plan(fm, **kw):
    a = dict(PLAN, B=3, N=10, Bt=4, mp=8, n=20, P=16)
    a.update(kw)
    return fm.lib().fmha_page_plan(a["sl"], a["nn"], a["bi"], a["tab"], a["free"], a["nf"], a["nfo"], a["slots"], a["pos"],
                                   a["cu"], a["ns"], a["B"], a["N"], a["Bt"], a["mp"], a["n"], a["P"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(N=-1), -1), (dict(P=0), -1), (dict(P=24), -1), (dict(P=256), -1), (dict(P=8), -1), (dict(Bt=0), -1),
    (dict(mp=0), -1), (dict(n=0), -1), (dict(B=0), -1), (dict(mp=(1 << 26) + 1), -1), (dict(n=1 << 27), -1),
    *[({x: None}, -1) for x in PLAN if x != "bi"], *[({x: PLAN[x] + 2}, -1) for x in PLAN],
    (dict(B=8193), -2), (dict(B=0, N=0, sl=None), 0),
])
def test_plan_refusals(fm, kw, code):
    assert call_plan(fm, **kw) == code


def test_plan_outputs_over_inputs_and_one_another(fm, no_device):
    past = call_plan(fm)
    assert past not in (-1, 0)
    assert call_plan(fm, ns=PLAN["sl"]) == past and call_plan(fm, nfo=PLAN["nf"]) == past    # in place
    outs = ("tab", "free", "nfo", "slots", "pos", "cu", "ns")
    for i, x in enumerate(outs):
        for y in outs[i + 1:]:
            assert call_plan(fm, **{y: PLAN[x]}) == -1, (x, y)
            assert call_plan(fm, **{y: PLAN[x] + PLAN_BYTES[x] - 4}) == -1, (x, y)
            assert call_plan(fm, **{y: PLAN[x] + PLAN_BYTES[x]}) == past, (x, y)
        for y in ("sl", "nn", "bi", "nf"):
            if (x, y) not in (("ns", "sl"), ("nfo", "nf")):
                assert call_plan(fm, **{x: PLAN[y]}) == -1, (x, y)
    assert call_plan(fm, ns=PLAN["sl"] + 4) == -1        # not the lengths themselves


# ---------------------------------------------------------------------------
# Write: 5 tokens of 2 heads, 6 pages of 32
# ---------------------------------------------------------------------------

WRITE = apart("k", "v", "slots", "kp", "vp", "ks", "vs")
PAGE_BYTES, SCALE_BYTES = 6 * 2 * 32 * 128, 6 * 2 * 4


def call_write(fm, **kw):
    a = dict(WRITE, N=5, H_k=2, D=128, n=6, P=32, kt=256, kh=128, vt=256, vh=128, dt=BF16)
    a.update(kw)
    t = lambda x, d: fm.fmha_tensor(a[x], a.get(x + "_dt", d))
    return fm.lib().fmha_page_write(t("k", a["dt"]), a["kt"], a["kh"], t("v", a["dt"]), a["vt"], a["vh"], a["slots"],
                                    a["kp"], a["vp"], a["ks"], a["vs"], a["N"], a["H_k"], a["D"], a["n"],
                                    a["P"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), -1), (dict(H_k=0), -1), (dict(D=64), -1), (dict(P=48), -1), (dict(n=0), -1), (dict(n=1 << 26), -1),
    (dict(H_k=65536), -1), (dict(kt=-8), -1), (dict(vh=1 << 41), -1), (dict(kt=260), -2), (dict(vh=4), -2),
    *[({x: None}, -1) for x in WRITE], *[({x: WRITE[x] + 8}, -2) for x in ("k", "v", "kp", "vp")],
    *[({x: WRITE[x] + 2}, -1) for x in ("slots", "ks", "vs")],
    (dict(dt=E4M3), -2), (dict(v_dt=F16), -2), (dict(dt=7), -2),
    (dict(N=0, k=None, slots=None), 0),
])
def test_write_refusals(fm, kw, code):
    assert call_write(fm, **kw) == code


def test_write_cache_over_inputs_and_itself(fm, no_device):
    past = call_write(fm)
    assert past not in (-1, 0)
    assert call_write(fm, v=WRITE["k"]) == past          # both are only read
    size = dict(k=5 * 512, v=5 * 512, slots=20, kp=PAGE_BYTES, vp=PAGE_BYTES, ks=SCALE_BYTES, vs=SCALE_BYTES)
    for x in ("kp", "vp", "ks", "vs"):
        for y in WRITE:
            if x != y:
                assert call_write(fm, **{y: WRITE[x]}) == -1, (x, y)
                if size[x] >= 16:
                    assert call_write(fm, **{y: WRITE[x] + size[x] - 16}) == -1, (x, y)
                assert call_write(fm, **{y: WRITE[x] + size[x]}) == past, (x, y)


# ---------------------------------------------------------------------------
# Rope: [2, 5, 4 (2), 64]
# ---------------------------------------------------------------------------

ROPE = apart("q", "k", "qo", "ko", "pos", "f")


def call_rope(fm, **kw):
    a = dict(ROPE, B=2, S=5, H=4, H_k=2, D=64, rot=64, m=1.0, layout=0, tr=0, dt=BF16, odt=None,
             qs=(1280, 256, 64), ks=(640, 128, 64), qos=(1280, 256, 64), kos=(640, 128, 64))
    a.update(kw)
    odt = a["dt"] if a["odt"] is None else a["odt"]
    t = lambda x, d: fm.fmha_tensor(a[x], a.get(x + "_dt", d))
    return fm.lib().fmha_rope(t("q", a["dt"]), *a["qs"], t("k", a["dt"]), *a["ks"], t("qo", odt), *a["qos"],
                              t("ko", odt), *a["kos"], a["B"], a["S"], a["H"], a["H_k"], a["D"], a["rot"], a["pos"], a["f"],
                              a["m"], a["layout"], a["tr"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(S=-1), -1), (dict(H=-1), -1), (dict(H_k=-1), -1), (dict(D=0), -1), (dict(D=258, rot=2), -1), (dict(rot=0), -1),
    (dict(rot=66), -1), (dict(rot=33), -1), (dict(layout=2), -1), (dict(m=float("nan")), -1), (dict(m=float("inf")), -1),
    (dict(f=None), -1), (dict(f=ROPE["f"] + 4), -1), (dict(pos=ROPE["pos"] + 2), -1), (dict(H=65535), -1),
    *[({x: None}, -1) for x in ("q", "k", "qo", "ko")], *[({x: ROPE[x] + 1}, -2) for x in ("q", "k", "qo", "ko")],
    (dict(dt=E4M3), -2), (dict(k_dt=F16), -2), (dict(odt=F16), -2), (dict(ko_dt=E4M3), -2), (dict(dt=9), -2),
    (dict(B=1 << 16, S=1 << 15), -1), (dict(qs=(1280, 256, -64)), -1), (dict(qos=(1280, 256, 0)), -1), (dict(qos=(1280, 255, 64)), -1),
    (dict(qos=(1279, 256, 64)), -1), (dict(kos=(0, 128, 64)), -1), (dict(qos=(64, 64, 64)), -1),
    (dict(B=0, q=None), 0), (dict(S=0, f=None), 0), (dict(H=0, H_k=0), 0),
])
def test_rope_refusals(fm, kw, code):
    assert call_rope(fm, **kw) == code


def test_rope_outputs_over_inputs(fm, no_device):
    past = call_rope(fm)
    assert past not in (-1, 0)
    R = ROPE
    assert call_rope(fm, qo=R["q"], ko=R["k"]) == past                            # in place
    assert call_rope(fm, H_k=0, k=None, ko=None) == past and call_rope(fm, H=0, q=None, qo=None) == past
    assert call_rope(fm, pos=None) == past
    for x, y, n in (("q", "ko", 2560), ("k", "qo", 1280), ("qo", "ko", 2560), ("qo", "pos", 2560), ("ko", "f", 1280), ("qo", "k", 2560)):
        assert call_rope(fm, **{y: R[x]}) == -1, (x, y)
        assert call_rope(fm, **{y: R[x] + n * 2 - 16}) == -1, (x, y)
        assert call_rope(fm, **{y: R[x] + n * 2}) == past, (x, y)
    assert call_rope(fm, qo=R["q"] + 128) == -1                                   # over its own input, shifted
    assert call_rope(fm, qo=R["q"], qos=(1280, 64, 320)) == -1                    # other strides
    assert call_rope(fm, qo=R["q"], odt=E4M3) == -1                               # other element size
    # pieces of one projection's rows [2, 5, (4 + 2 + 2) * 64]
    row = dict(qs=(2560, 512, 64), ks=(2560, 512, 64), qos=(2560, 512, 64), kos=(2560, 512, 64))
    k = R["q"] + 4 * 64 * 2
    assert call_rope(fm, **row, k=k, qo=R["q"], ko=k) == past
    assert call_rope(fm, **row, k=k - 2, qo=R["q"], ko=k - 2) == -1               # one element in common
    assert call_rope(fm, **row, k=k + 2 * 512, qo=R["q"], ko=k + 2 * 512) == past # a token further on
    # q's heads, and in another layout head by head: interleaved spans that are not pieces of tokens
    assert call_rope(fm, qo=R["q"] + 2, qos=(1280, 256, 64)) == -1


# ---------------------------------------------------------------------------
# Attention: 3 sequences, 7 rows, 8 heads on 2, 6 pages of 32, a table of 4 rows of 5
# ---------------------------------------------------------------------------

FWD = apart("q", "kp", "vp", "ks", "vs", "o", "lse", "tab", "sl", "bi", "cu", "ws")


def call_fwd(fm, **kw):
    a = dict(FWD, B=3, N=7, mq=4, H=8, H_k=2, D=128, n=6, P=32, Bt=4, mp=5, scale=0.1, out_scale=1.0, mask=2, ws_bytes=1 << 30, dt=BF16)
    a.update(kw)
    t = lambda x: fm.fmha_tensor(a[x], a.get(x + "_dt", a["dt"]))
    return fm.lib().fmha_page_fwd(t("q"), a["kp"], a["vp"], a["ks"], a["vs"], t("o"), a["lse"], a["B"], a["N"], a["mq"], a["H"],
                                  a["H_k"], a["D"], a["n"], a["P"], a["Bt"], a["mp"], a["tab"], a["sl"], a["bi"], a["cu"],
                                  a["scale"], a["out_scale"], a["mask"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(N=-1), -1), (dict(D=64), -1), (dict(H=3), -1), (dict(H=258, H_k=2), -1), (dict(H_k=0), -1),
    (dict(P=8), -1), (dict(P=100), -1), (dict(P=0), -1), (dict(P=256), -1), (dict(mq=0), -1), (dict(n=0), -1), (dict(Bt=0), -1), (dict(mp=0), -1),
    (dict(mp=(1 << 25) + 1), -1), (dict(n=1 << 26), -1), (dict(N=1 << 28), -1), (dict(cu=None), -1),
    (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(out_scale=float("inf")), -1),
    (dict(out_scale=float("nan")), -1), (dict(mask=1), -1), (dict(mask=3), -1), (dict(ws=None), -1), (dict(ws=FWD["ws"] + 128), -1),
    (dict(ws_bytes=1000), -1), *[({x: None}, -1) for x in ("q", "kp", "vp", "ks", "vs", "o", "tab", "sl")],
    *[({x: FWD[x] + 8}, -2) for x in ("q", "kp", "vp", "o")],
    *[({x: FWD[x] + 2}, -1) for x in ("ks", "vs", "lse", "tab", "sl", "bi", "cu")],
    (dict(dt=E4M3), -2), (dict(o_dt=F16), -2), (dict(dt=8), -2),
    (dict(B=0, q=None, ws=None), 0), (dict(N=0, q=None, ws=None), 0),
])
def test_fwd_refusals(fm, kw, code):
    assert call_fwd(fm, **kw) == code


def test_fwd_outputs_over_inputs_and_one_another(fm, no_device):
    past = call_fwd(fm)
    assert past not in (-1, 0)
    assert call_fwd(fm, N=3, cu=None) == past and call_fwd(fm, bi=None, lse=None) == past
    assert call_fwd(fm, vp=FWD["kp"], vs=FWD["ks"]) == past                       # both are only read
    rows, ws = 7 * 8 * 256, fm.fmha_page_workspace_size(4, 8, 2)
    size = dict(q=rows, kp=PAGE_BYTES, vp=PAGE_BYTES, ks=SCALE_BYTES, vs=SCALE_BYTES, o=rows, lse=7 * 8 * 4, tab=80, sl=12, bi=12,
                cu=16, ws=ws)
    for x in ("o", "lse", "ws"):
        for y in FWD:
            if x == y:
                continue
            assert call_fwd(fm, **{y: FWD[x]}) == -1, (x, y)
            end = FWD[x] + (size[x] + 255) // 256 * 256
            assert call_fwd(fm, **{y: end}) == past, (x, y)
            if size[x] > 16 and y != "ws":
                assert call_fwd(fm, **{y: FWD[x] + size[x] - 16}) == -1, (x, y)


def test_page_workspace_size(fm):
    size = fm.fmha_page_workspace_size
    row, meta = (128 + 1) * 4, 16
    for max_q, H, H_k, rows in ((1, 32, 8, 16), (4, 32, 8, 16), (5, 32, 8, 32), (8, 32, 8, 32), (9, 32, 8, 128), (32, 32, 8, 128), (33, 32, 8, 128),
                                (1, 128, 1, 128), (2, 128, 1, 128), (1, 33, 1, 128), (1000, 8, 8, 128)):
        assert size(max_q, H, H_k) == 2 * 152 * (rows * row + meta)
    assert size(1000, 8, 8) <= 20_100_000
    for bad in ((0, 8, 8), (1, 8, 3), (1, 129, 1), (1, 0, 1), (1, 8, 0), (-1, 8, 8)):
        assert size(*bad) == 0
