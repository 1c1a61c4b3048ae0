"""How the cache operators are called: refusals of the Python entry points,
streams, an expired wait, and rows around what a call may write."""
import pytest
import torch

from tests import cache_util as cu
from tests import test_cache_gpu as tc
from tests import test_tree_gpu as tt

pytestmark = pytest.mark.gpu
i32 = tc.i32


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_attention_forward_02_gb300 import build, fmha
    build.build()
    fmha.lib()
    return fmha


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


TREE = dict(q=(2, 3, 4, 128), k_cache=(2, 8, 2, 128), v_cache=(2, 8, 2, 128), k_new=(2, 3, 2, 128), v_new=(2, 3, 2, 128))


@pytest.mark.parametrize("name,bad", [
    ("v_cache", lambda: bf(2, 7, 2, 128)), ("k_new", lambda: bf(2, 4, 2, 128)), ("k_new", lambda: bf(2, 3, 2, 128).half()),
    ("k_cache", lambda: bf(2, 2, 8, 128).transpose(1, 2)), ("q", lambda: bf(2, 3, 4, 256)[..., ::2]),
    ("seqlen", lambda: i32([1])), ("seqlen", lambda: i32([1, 1]).long()), ("n_draft", lambda: i32([1, 1, 1])),
    ("batch_idx", lambda: i32([0, 1]).cpu()), ("tree_mask", lambda: torch.ones((3, 4), dtype=torch.bool, device="cuda")),
    ("tree_mask", lambda: torch.ones((1, 3, 3), dtype=torch.bool, device="cuda")),
    ("tree_mask", lambda: torch.ones((3, 3), dtype=torch.int32, device="cuda")), ("out", lambda: bf(2, 3, 4, 64)),
    ("lse", lambda: torch.zeros((2, 3, 4), device="cuda")), ("workspace", lambda: torch.zeros(1 << 22)),
])
def test_tree_refuses_tensors_that_it_would_misread(fm, name, bad):
    a = {k: bf(*s) for k, s in TREE.items()}
    a.update(seqlen=i32([4, 4]))
    kw = {"n_draft": None, "batch_idx": None, "tree_mask": None, "out": None, "lse": None, "workspace": None}
    (a if name in a else kw)[name] = bad()
    with pytest.raises(ValueError):
        fm.tree_fwd(*a.values(), **kw)


def test_other_refusals(fm):
    kc, kn, sl = bf(2, 8, 2, 128), bf(2, 3, 2, 128), i32([4, 4])
    q, lse, acc = bf(2, 3, 4, 128), torch.zeros((2, 4, 3), device="cuda"), torch.zeros((2, 2, 8), device="cuda")
    path = i32([[0], [1]])
    calls = [
        lambda: fm.tree_commit(kc, kc[:1], kn, kn, sl, path, i32([1, 1])),
        lambda: fm.tree_commit(kc, kc, kn, kn.half(), sl, path, i32([1, 1])),
        lambda: fm.tree_commit(kc, kc, kn, kn, sl, path.long(), i32([1, 1])),
        lambda: fm.tree_commit(kc, kc, kn, kn, sl, path[0], i32([1, 1])),
        lambda: fm.cache_weights(q, kc, lse.transpose(1, 2), sl),
        lambda: fm.cache_weights(q, kc, lse.double(), sl),
        lambda: fm.cache_weights(q, kc, lse, sl, acc=acc[:, :1]),
        lambda: fm.cache_weights(q, kc, lse, sl, mask="residual"),
        lambda: fm.cache_weights(q[0, 0], kc, lse, sl),
        lambda: fm.cache_evict(kc, kc.clone(), acc, sl, 4, k_out=kc.clone()),
        lambda: fm.cache_evict(kc, kc.clone(), acc, sl, 4, out_idx=i32([0, 1])),
        lambda: fm.cache_evict(kc, kc.clone(), acc.half(), sl, 4),
        lambda: fm.cache_evict(kc, kc.clone(), acc, sl, 4, kept=i32([[1]])),
    ]
    for i, c in enumerate(calls):
        with pytest.raises(ValueError):
            c()
    for c in (lambda: fm.cache_evict(kc, kc.clone(), acc, sl, 0), lambda: fm.cache_evict(kc, kc.clone(), acc, sl, 9),
              lambda: fm.cache_evict(kc, kc.clone(), acc, sl, 4, recent=5),
              lambda: fm.cache_evict(kc, kc.clone(), acc, sl, 4, new_seqlen=sl),
              lambda: fm.tree_fwd(q.float(), kc, kc, kn, kn, sl),
              lambda: fm.tree_fwd(q, kc, kc, kn, kn, sl, workspace=torch.zeros(100, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fm.FmhaError):
            c()


def test_empty_calls(fm):
    kc, acc = bf(2, 8, 2, 128), torch.ones((2, 2, 8), device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    o, lse = fm.tree_fwd(bf(0, 3, 4, 128), kc, kc, bf(0, 3, 2, 128), bf(0, 3, 2, 128), none)
    assert o.shape == (0, 3, 4, 128) and lse.shape == (0, 4, 3)
    o, lse = fm.tree_fwd(bf(2, 0, 4, 128), kc, kc, bf(2, 0, 2, 128), bf(2, 0, 2, 128), i32([1, 2]))
    assert o.shape == (2, 0, 4, 128)
    fm.tree_commit(kc, kc, bf(0, 3, 2, 128), bf(0, 3, 2, 128), none, none.view(0, 4), none)
    assert fm.cache_weights(bf(2, 0, 4, 128), kc, torch.zeros((2, 4, 0), device="cuda"), i32([1, 2]), acc=acc) is acc
    fm.cache_evict(kc, kc.clone(), acc, none, 3)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0 and bool((acc == 1).all())


def test_work_on_another_stream_than_the_current_one(fm):
    """Inputs written on a side stream just before the call, which runs there; the current stream does other work."""
    c = tt.make("bf16", 9, 8, 2, 3000, [2999, 1500], seed=21)
    side = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(10):
            x = x @ x * 1e-3                              # the copies below come late
        d = tt.on_gpu(c)
        o, lse = tt.outputs(c)
    ws = torch.empty(fm.fmha_tree_workspace_size(2, 9, 8, 2, 128, 3000), dtype=torch.uint8, device="cuda")
    fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse, workspace=ws, stream=side)
    acc = torch.zeros((2, 2, 3000), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fm.cache_weights(d["args"][0], d["args"][1], lse, d["args"][5], acc=acc)
        kept, new = fm.cache_evict(d["args"][1], d["args"][2], acc, d["args"][5], 1000, recent=10)
    side.synchronize()
    assert fm.device_status(reset=True) == 0
    tt.check(c, o, lse)
    assert new.tolist() == [1000, 1000] and bool((kept[:, :, 1:] > kept[:, :, :-1]).all())


@pytest.mark.parametrize("handle", [False, True])
def test_what_a_call_makes_for_itself_belongs_to_its_stream(fm, handle):
    """The current stream is busy: a zero fill or a workspace left to it would come after, or under, the kernels."""
    c = tc.make("bf16", 40, 8, 2, 900, [900, 301], mask="causal", seed=22)
    c["want"] -= c["acc"].double()                        # from nothing
    t = tt.make("bf16", 40, 8, 2, 900, [900, 301], seed=23)
    args = c["q"].cuda(), c["kc"].cuda(), c["lse"].cuda(), i32(c["seqlen"])
    d = tt.on_gpu(t)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    for _ in range(2):                                    # the kernels are loaded before the streams part
        fm.cache_weights(*args, mask="causal", stream=stream)
        fm.tree_fwd(*d["args"], **d["kw"], stream=stream)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    r = fm.cache_weights(*args, mask="causal", stream=stream)
    o, lse = fm.tree_fwd(*d["args"], **d["kw"], stream=stream)
    side.synchronize()
    assert not torch.cuda.current_stream().query()        # none of it waited for the current stream
    torch.full((1 << 22,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    tc.check_weights(c, r, torch.zeros_like(c["acc"]))
    tt.check(t, o, lse)


@pytest.mark.parametrize("op", ["tree", "weights"])
def test_scratch_of_a_captured_call_stays_its_own(fm, op):
    """What the call took from the allocator belongs to the graph: later tensors get none of it."""
    if op == "tree":
        c = tt.make("bf16", 70, 8, 2, 3000, [2900, 1501], seed=24)
        d, (o, lse) = tt.on_gpu(c), tt.outputs(c)
        size = fm.fmha_tree_workspace_size(2, 70, 8, 2, 128, 3000)
        run = lambda: fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse)
        check = lambda: tt.check(c, o, lse)
    else:
        c = tc.make("bf16", 140, 8, 2, 1500, [1500, 701], mask="causal", seed=25)
        args = c["q"].cuda(), c["kc"].cuda(), c["lse"].cuda(), i32(c["seqlen"])
        acc, o = c["acc"].cuda(), torch.zeros(c["acc"].shape, device="cuda")
        size = fm.fmha_cache_weights_workspace_size()
        run = lambda: fm.cache_weights(*args, mask="causal", acc=acc, out=o)
        check = lambda: tc.check_weights(c, o, torch.zeros_like(c["acc"]))
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    later = [torch.full((size,), 0x5a, dtype=torch.uint8, device="cuda") for _ in range(8)]
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    assert all(bool((t == 0x5a).all()) for t in later)
    check()


def test_an_output_over_an_input_is_refused(fm):
    a = {k: bf(*s) for k, s in TREE.items()}
    with pytest.raises(fm.FmhaError):
        fm.tree_fwd(*a.values(), i32([4, 4]), out=a["q"])
    with pytest.raises(fm.FmhaError):
        fm.tree_commit(a["k_cache"], a["k_cache"], a["k_new"], a["v_new"], i32([4, 4]), i32([[0], [0]]), i32([1, 1]))


@pytest.mark.parametrize("op", ["tree_blocks", "tree_split", "weights"])
def test_expired_wait_is_reported_and_the_context_stays_usable(fm, op):
    """With the bounded waits limited to 1 ms the producers first wait for a
    flag that nothing sets: the call reports it, and the next one is right."""
    if op == "weights":
        c = tc.make("bf16", 70, 8, 2, 1500, [1500, 700, 0], mask="causal", seed=31)
        out = torch.zeros(c["acc"].shape, device="cuda")
        run = lambda: tc.weights(fm, c, acc=c["acc"].cuda(), out=out)
        check = lambda r: tc.check_weights(c, r, torch.zeros_like(c["acc"]))
    else:
        c = tt.make("bf16", 40 if op == "tree_blocks" else 6, 16, 4, 1500, [1500, 700, 0], seed=32)
        d = tt.on_gpu(c)
        run = lambda: fm.tree_fwd(*d["args"], **d["kw"])
        check = lambda r: tt.check(c, *r)
    assert fm.device_status(reset=True) == 0
    assert fm.set_wait_limit_ns(1_000_000) == 0
    assert fm.set_test_gate(True) == 0
    try:
        run()
        torch.cuda.synchronize()
        status = fm.device_status(reset=True)
    finally:
        assert fm.set_test_gate(False) == 0
        assert fm.set_wait_limit_ns(0) == 0
    assert status == fm.ERR_TIMEOUT
    if op == "weights":
        out.zero_()
    r = run()
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    check(r)


def guarded(t, pad=1024):
    """A copy of t with sentinel bytes around it, and a check that they are still there."""
    n = t.numel() * t.element_size()
    buf = torch.full((n + 2 * pad,), cu.SENTINEL, dtype=torch.uint8, device="cuda")
    v = buf[pad:pad + n].view(t.dtype).view(t.shape)
    v.copy_(t)
    return v, lambda: bool((buf[:pad] == cu.SENTINEL).all()) and bool((buf[-pad:] == cu.SENTINEL).all())


def test_nothing_is_written_outside_the_outputs(fm):
    g = torch.Generator().manual_seed(41)
    c = tt.make("bf16", 37, 12, 4, 700, [700, 3, 129], n_draft=[37, 1, 36], seed=42)
    d = tt.on_gpu(c)
    (o, o_ok), (lse, l_ok) = (guarded(t) for t in tt.outputs(c))
    ws, w_ok = guarded(torch.zeros(fm.fmha_tree_workspace_size(3, 37, 12, 4, 128, 700), dtype=torch.uint8, device="cuda"))
    fm.tree_fwd(*d["args"], **d["kw"], out=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    tt.check(c, o, lse)
    assert o_ok() and l_ok() and w_ok()
    w = tc.make("f16", 130, 12, 4, 700, [700, 130, 501], mask="causal", seed=43)
    (acc, a_ok), (out, r_ok) = guarded(w["acc"].cuda()), guarded(torch.zeros(w["acc"].shape, device="cuda"))
    ws, w_ok = guarded(torch.zeros(fm.fmha_cache_weights_workspace_size(), dtype=torch.uint8, device="cuda"))
    tc.weights(fm, w, acc=acc, out=out, workspace=ws)
    torch.cuda.synchronize()
    tc.check_weights(w, out, torch.zeros_like(w["acc"]))
    assert a_ok() and r_ok() and w_ok()
    k, v = (cu.draw(g, (3, 333, 3, 128), "e4m3").cuda() for _ in range(2))
    acc, sl = torch.rand((3, 3, 333), generator=g).cuda(), i32([333, 100, 101])
    bufs = [guarded(t) for t in (torch.zeros((3, 101, 3, 128), dtype=torch.uint8, device="cuda").view(k.dtype),
                                 torch.zeros((3, 101, 3, 128), dtype=torch.uint8, device="cuda").view(k.dtype),
                                 torch.zeros((3, 3, 101), device="cuda"), torch.zeros((3, 3, 101), dtype=torch.int32, device="cuda"),
                                 torch.zeros((3,), dtype=torch.int32, device="cuda"))]
    fm.cache_evict(k, v, acc, sl, 101, recent=7, k_out=bufs[0][0], v_out=bufs[1][0], acc_out=bufs[2][0], kept=bufs[3][0],
                   new_seqlen=bufs[4][0])
    torch.cuda.synchronize()
    assert bufs[4][0].tolist() == [101, 100, 101]
    assert all(ok() for _, ok in bufs)


def test_offsets_past_32_bits(fm):
    """One entry of 2^31 elements behind another: every operator at its far end, against fp64 on the device."""
    S, H_k, H, T, e = 1 << 22, 4, 8, 2, 1
    g = torch.Generator(device="cuda").manual_seed(51)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.empty((2, S, H_k, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for c in (k, v):
        c[0].zero_()
        c[1].normal_(generator=g)
    q, kn, vn = rnd(1, T, H, 128), rnd(1, T, H_k, 128), rnd(1, T, H_k, 128)
    L, idx = S - T, i32([e])
    o, lse = fm.tree_fwd(q, k, v, kn, vn, i32([L]), batch_idx=idx)
    fm.tree_commit(k, v, kn, vn, i32([L]), i32([[0, 1]]), i32([T]), batch_idx=idx)
    assert torch.equal(k[e, L:], kn[0]) and torch.equal(v[e, L:], vn[0]) and not bool(k[0].any()) and not bool(v[0].any())
    acc = fm.cache_weights(q, k, lse, i32([S]), batch_idx=idx, mask="causal")
    assert fm.device_status(reset=True) == 0 and not bool(acc[0].any())
    see = torch.arange(S, device="cuda")[None, :] <= L + torch.arange(T, device="cuda")[:, None]
    for gg in (0, H_k - 1):
        keys, vals = k[e, :, gg].double(), v[e, :, gg].double()
        x = torch.einsum("thd,kd->thk", q[0, :, 2 * gg:2 * gg + 2].double(), keys) * 128 ** -0.5
        x = x.masked_fill(~see[:, None, :], float("-inf"))
        w = torch.softmax(x, -1)
        want = torch.einsum("thk,kd->thd", w, vals)
        # an average of 4 million values of size 1: every weight is rounded by up to 2^-8 of itself, independently of its
        # value's sign, and O once more
        err = (o[0, :, 2 * gg:2 * gg + 2].double() - want).abs()
        assert bool((err <= 2.0 ** -8 * torch.einsum("thk,kd->thd", w, vals.abs()) + 2.0 ** -8 * want.abs()).all())
        exact = torch.logsumexp(x, -1)
        assert bool(((lse[0, 2 * gg:2 * gg + 2].T.double() - exact).abs() <= 1e-4).all())
        # an exponential of an argument below 32 that is rounded a few times, 2^-18 in all, and the LSE above
        total = w.sum((0, 1))
        assert bool(((acc[e, gg].double() - total).abs() <= 2e-4 * total).all())
    budget, recent = 1000, 10
    ko, vo = (torch.zeros((1, budget, H_k, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ao = torch.zeros((1, H_k, budget), device="cuda")
    kept, new = fm.cache_evict(k, v, acc, i32([S]), budget, recent=recent, batch_idx=idx, k_out=ko, v_out=vo, acc_out=ao)
    assert fm.device_status(reset=True) == 0 and new.tolist() == [budget]
    for gg in range(H_k):
        top = torch.sort(acc[e, gg, :S - recent], descending=True, stable=True).indices[:budget - recent]
        rows = torch.cat([torch.sort(top).values, torch.arange(S - recent, S, device="cuda")])
        assert torch.equal(kept[0, gg].long(), rows) and torch.equal(ao[0, gg], acc[e, gg, rows])
        assert torch.equal(ko[0, :, gg], k[e, rows, gg]) and torch.equal(vo[0, :, gg], v[e, rows, gg])
