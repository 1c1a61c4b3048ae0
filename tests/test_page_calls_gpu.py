"""How the paged-cache operators are called: refusals of the Python entry points,
streams, an expired wait, guard bands, and values past 32-bit offsets."""
import pytest
import torch

from tests import cache_util as cu
from tests import page_util as pu
from tests import test_page_fwd_gpu as tf
from tests.test_page_fwd_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16, device="cuda")


def e4(*s):
    return torch.zeros(s, dtype=torch.uint8, device="cuda").view(pu.E4M3)


def f32(*s):
    return torch.zeros(s, device="cuda")


def test_refusals_of_tensors_that_would_be_misread(fm):  # noqa: F811
    pool = (e4(6, 2, 16, 128), e4(6, 2, 16, 128), f32(6, 2), f32(6, 2))
    q, table, sl = bf(3, 4, 128), i32([[0, 1], [2, 3], [4, 5]]), i32([1, 2, 3])
    swap = lambda i, t: [*pool[:i], t, *pool[i + 1:]]
    new, slots = bf(3, 2, 128), i32([0, 16, 32])
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    plan = lambda **kw: fm.page_plan(**{**dict(seqlen=sl, n_new=sl, table=table, free_list=i32([0] * 6), n_free=i32([0]), page_size=16,
                                               max_tokens=6), **kw})
    calls = [
        *[lambda i=i: fm.page_fwd(q, *swap(i, e4(6, 2, 32, 128)[:, :, ::2]), table, sl) for i in (0, 1)],
        lambda: fm.page_fwd(q, *swap(1, e4(6, 2, 32, 128)), table, sl), lambda: fm.page_fwd(q, *swap(2, f32(6, 1)), table, sl),
        lambda: fm.page_fwd(q, *swap(3, f32(6, 2).double()), table, sl), lambda: fm.page_fwd(q, *swap(0, bf(6, 2, 16, 128)), table, sl),
        lambda: fm.page_fwd(q, *pool, table.long(), sl), lambda: fm.page_fwd(q, *pool, table, sl[:2]),
        lambda: fm.page_fwd(q, *pool, table, sl, cu_q=i32([0, 1, 2])), lambda: fm.page_fwd(q[:, ::2], *pool, table, sl),
        lambda: fm.page_fwd(q, *pool, table, sl, batch_idx=i32([0, 1])), lambda: fm.page_fwd(q, *pool, table, sl, out=bf(3, 4, 64)),
        lambda: fm.page_fwd(q, *pool, table, sl, lse=f32(4, 3)), lambda: fm.page_fwd(q, *pool, table, sl.cpu()),
        lambda: fm.page_fwd(q, *pool, table, sl, mask="residual"), lambda: fm.page_fwd(q[0], *pool, table, sl),
        lambda: fm.page_fwd(q, *pool, table, sl, workspace=torch.zeros(1 << 23)),
        lambda: fm.page_write(new, new[:2], slots, *pool), lambda: fm.page_write(new, new.half(), slots, *pool),
        lambda: fm.page_write(new, bf(3, 2, 256)[..., ::2], slots, *pool), lambda: fm.page_write(new, new, slots[:2], *pool),
        lambda: fm.page_write(new, new, slots.long(), *pool), lambda: fm.page_write(new, new, slots, *swap(3, f32(2, 6).T)),
        lambda: plan(n_new=sl[:2]), lambda: plan(n_new=sl.long()), lambda: plan(table=table.T), lambda: plan(n_free=i32([0, 0])),
        lambda: plan(batch_idx=i32([0, 1])), lambda: plan(slots=i32([0] * 5)), lambda: plan(cu_new=sl), lambda: plan(max_tokens=None),
        lambda: plan(free_list=i32([0] * 12)[::2]), lambda: plan(seqlen=sl.cpu()),
        lambda: fm.rope(q, None, f.float()), lambda: fm.rope(q, bf(2, 2, 128), f), lambda: fm.rope(q, bf(3, 2, 64), f),
        lambda: fm.rope(q, None, f, positions=i32([0, 1])), lambda: fm.rope(q, None, f, positions=i32([0, 1, 2]).long()),
        lambda: fm.rope(q, None, f, q_out=bf(3, 4, 256)[..., ::2]), lambda: fm.rope(q, None, f, k_out=q), lambda: fm.rope(q[0], None, f),
        lambda: fm.rope(q, None, f.cpu()), lambda: fm.rope_frequencies(7), lambda: fm.rope_frequencies(8, scaling="other"),
        lambda: fm.rope_frequencies(8, scaling="by_parts", factor=2.0), lambda: fm.rope_frequencies(8, factor=0.5),
    ]
    for i, c in enumerate(calls):
        with pytest.raises(ValueError):
            c()
            pytest.fail(f"call {i} was not refused")
    for i, c in enumerate((lambda: fm.page_fwd(q.float(), *pool, table, sl), lambda: fm.page_write(new.float(), new.float(), slots, *pool),
                           lambda: fm.rope(q, None, f, out_dtype=torch.float32), lambda: fm.rope(q, None, torch.cat([f, f, f])),
                           lambda: fm.page_fwd(q, *pool, table, sl, workspace=torch.zeros(100, dtype=torch.uint8, device="cuda")),
                           lambda: plan(page_size=8), lambda: plan(new_seqlen=sl, n_new=sl))):
        with pytest.raises(fm.FmhaError):
            c()
            pytest.fail(f"call {i} was not refused")


def test_empty_calls(fm):  # noqa: F811
    pool = (e4(6, 2, 16, 128), e4(6, 2, 16, 128), f32(6, 2), f32(6, 2))
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    o, lse = fm.page_fwd(bf(0, 4, 128), *pool, torch.zeros((1, 2), dtype=torch.int32, device="cuda"), none)
    assert o.shape == (0, 4, 128) and lse.shape == (0, 4)
    fm.page_write(bf(0, 2, 128), bf(0, 2, 128), none, *pool)
    q, k = fm.rope(bf(0, 4, 64), bf(0, 2, 64), torch.ones(16, dtype=torch.float64, device="cuda"))
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    slots, pos, cu_new, new = fm.page_plan(i32([5]), i32([0]), i32([[3]]), i32([0] * 4), i32([0]), page_size=16, max_tokens=0)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0 and cu_new.tolist() == [0, 0] and new.tolist() == [5]


def late(side):
    """Work that keeps a stream busy for a while."""
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)


@pytest.mark.parametrize("handle", [False, True])
def test_all_run_on_the_given_stream(fm, handle):  # noqa: F811
    """Their inputs come late on a side stream; nothing of them runs on the current one."""
    c = tf.make("bf16", 8, 2, 32, [700, 300], [3, 1], seed=30)
    d, (o, lse) = tf.on_gpu(c), tf.outputs(c)
    q, table = d["args"][0].clone(), d["args"][5].clone()
    fm.page_fwd(*d["args"], **d["kw"])                    # the kernel is loaded before the streams part
    f, _ = fm.rope_frequencies(64, device="cuda")
    x, y = bf(50, 3, 64), bf(50, 3, 64)
    fm.rope(x, None, f, q_out=y)
    d["args"][0].zero_()
    d["args"][5].zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late(side)
    with torch.cuda.stream(side):
        d["args"][0].copy_(q)
        d["args"][5].copy_(table)
        x.fill_(1.0)
    s = side.cuda_stream if handle else side
    fm.page_fwd(*d["args"], **d["kw"], out=o, lse=lse, stream=s)
    fm.rope(x, None, f, q_out=y, positions=None, stream=s)
    # kept until the side stream is past them: their memory is the current stream's
    seqlen, n_new, tab, free, n_free = i32([16]), i32([1]), i32([[3, 0]]), i32([1, 2, 0, 0]), i32([2])
    pool, k, v = (e4(4, 1, 16, 128), e4(4, 1, 16, 128), f32(4, 1), f32(4, 1)), bf(1, 1, 128), bf(1, 1, 128)
    slots, pos, _, new = fm.page_plan(seqlen, n_new, tab, free, n_free, page_size=16, max_tokens=1, stream=s)
    fm.page_write(k, v, slots, *pool, stream=s)
    assert not side.query()
    side.synchronize()
    assert fm.device_status(reset=True) == 0
    tf.check(c, o, lse)
    assert slots.tolist() == [32] and new.tolist() == [17] and pool[2][2, 0].item() == 2.0 ** -60
    assert y[0, 0, 0].item() == 1.0 and y.abs().sum().item() > 0


def test_the_default_stream_by_its_handle(fm):  # noqa: F811
    c = tf.make("f16", 8, 2, 32, [700, 300], seed=31)
    d, (o, lse) = tf.on_gpu(c), tf.outputs(c)
    fm.page_fwd(*d["args"], **d["kw"])
    q = d["args"][0].clone()
    d["args"][0].zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    d["args"][0].copy_(q)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fm.page_fwd(*d["args"], **d["kw"], out=o, lse=lse, stream=0)
    assert side.query() and not torch.cuda.default_stream().query()
    torch.cuda.synchronize()
    tf.check(c, o, lse)


@pytest.mark.parametrize("news", [None, [3, 1], [20, 10], [200, 60]])
def test_nothing_around_the_outputs_and_the_workspace_is_written(fm, news):  # noqa: F811
    c = tf.make("bf16", 8, 2, 32, [900, 333], news, seed=32)
    d = tf.on_gpu(c)
    (N, H, D), pad = c["q"].shape, 4096
    need = fm.fmha_page_workspace_size(d["kw"]["max_q"], H, 2)
    raw = [cu.sentinel((n + 2 * pad,), torch.uint8) for n in (N * H * D * 2, N * H * 4, need)]
    o, lse, ws = (r[pad:-pad] for r in raw)
    o, lse = o.view(torch.bfloat16).view(N, H, D), lse.view(torch.float32).view(N, H)
    before = [t.view(torch.uint8).clone() for t in d["args"]]
    fm.page_fwd(*d["args"], **d["kw"], out=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    tf.check(c, o, lse)
    assert all(cu.untouched(r[:pad]) and cu.untouched(r[-pad:]) for r in raw)
    assert all(torch.equal(t.view(torch.uint8), b) for t, b in zip(d["args"], before))


@pytest.mark.parametrize("news", [None, [6, 7], [120, 200]])
def test_an_expired_wait_is_reported_and_the_next_call_is_right(fm, news):  # noqa: F811
    c = tf.make("bf16", 8, 2, 64, [3000, 2000], news, seed=33)
    assert fm.device_status(reset=True) == 0
    assert fm.set_wait_limit_ns(1_000_000) == 0 and fm.set_test_gate(True) == 0
    try:
        _, _, status = tf.run(fm, c)
    finally:
        assert fm.set_test_gate(False) == 0 and fm.set_wait_limit_ns(0) == 0
    assert status == fm.ERR_TIMEOUT
    o, lse, status = tf.run(fm, c)
    assert status == 0
    tf.check(c, o, lse)


@pytest.mark.parametrize("news", [None, [150, 1]])
def test_values_past_32_bits(fm, news):  # noqa: F811
    """Pages whose bytes lie past 2^32 in both pools, behind pages of zeros; written and read."""
    P, H_k, H, n_pages = 64, 8, 16, 70000                 # 4.6e9 bytes a pool
    pool = [torch.zeros((n_pages, H_k, P, 128), dtype=torch.uint8, device="cuda").view(pu.E4M3) for _ in range(2)] + \
        [torch.zeros((n_pages, H_k), device="cuda") for _ in range(2)]
    g = torch.Generator().manual_seed(34)
    lengths = [700, 100]
    ids = [[n_pages - 1 - 3 * i for i in range(11)], [n_pages - 2, n_pages - 5]]
    slots = [ids[b][i // P] * P + i % P for b in (0, 1) for i in range(lengths[b])]
    k, v = (torch.randn((800, H_k, 128), generator=g).to(torch.bfloat16) for _ in range(2))
    v += 1.0                                              # a mean: lost or wrapped loads show
    fm.page_write(k.cuda(), v.cuda(), i32(slots), *pool)
    n = news or [1, 1]
    q = torch.randn((sum(n), H, 128), generator=g).to(torch.bfloat16)
    table = i32([ids[0], ids[1] + [-1] * 9])
    cu_q = i32([0, n[0], n[0] + n[1]]) if news else None
    o, lse = fm.page_fwd(q.cuda(), *pool, table, i32(lengths), cu_q=cu_q, max_q=max(n))
    torch.cuda.synchronize()
    assert fm.device_status(reset=True) == 0
    near = torch.tensor(sum(ids, []))
    c = dict(dtype="bf16", H=H, H_k=H_k, P=P, L=lengths, n=n, entries=[0, 1], mask="causal", q=q,
             table=torch.tensor([list(range(11)), [11, 12] + [-1] * 9], dtype=torch.int32))
    for x, i in (("k", 0), ("v", 1)):
        c[x + "c"], c[x + "s"] = pool[i].view(torch.uint8)[near.cuda()].cpu().view(pu.E4M3), pool[2 + i][near.cuda()].cpu()
    want = v[:700].double()
    got = pu.VALUES[c["vc"].view(torch.uint8)[:11].long()] * c["vs"][:11].double()[..., None, None]
    got = got.transpose(1, 2).reshape(-1, H_k, 128)[:700]
    assert bool(((got - want).abs() <= want.abs() * 2.0 ** -4 + 2.0 ** -9).all())
    tf.check(c, o, lse)
    assert all(int(torch.count_nonzero(p.view(torch.uint8)[:n_pages - 40])) == 0 for p in pool[:2])


def test_turns_past_32_bits(fm):  # noqa: F811
    """Elements past 2^31 of a packed tensor, in place, and by a stride."""
    S, H, D = 300_000, 64, 128
    x = torch.empty((S, H, D), dtype=torch.bfloat16, device="cuda").normal_()
    f, _ = fm.rope_frequencies(D, device="cuda")
    pick = torch.tensor([0, 1, S // 2, 262143, 262144, 262145, S - 1])
    was = x[pick.cuda()].cpu()
    fm.rope(x, None, f, q_out=x)
    y, tol = pu.rope(was, f.cpu(), pick, False, 1.0)
    cu.close(x[pick.cuda()].double().cpu(), y, tol + (y.abs() + tol) * 2.0 ** -8, "turned rows")


@pytest.mark.parametrize("name", ["fwd", "rope", "write", "plan"])
def test_calls_without_allocation(fm, name):  # noqa: F811
    """With outputs and workspace given, torch's allocator is not asked."""
    c = tf.make("bf16", 8, 2, 32, [300, 200], seed=35)
    d, (o, lse) = tf.on_gpu(c), tf.outputs(c)
    ws = torch.empty(fm.fmha_page_workspace_size(1, 8, 2), dtype=torch.uint8, device="cuda")
    f, _ = fm.rope_frequencies(128, device="cuda")
    k, slots = bf(2, 2, 128), i32([5, 40])
    p = dict(seqlen=i32([0]), n_new=i32([1]), table=i32([[0]]), free_list=i32([1, 0]), n_free=i32([1]), page_size=16, slots=i32([0]),
             positions=i32([0]), cu_new=i32([0, 0]), new_seqlen=i32([0]), n_free_out=i32([0]))
    call = dict(fwd=lambda: fm.page_fwd(*d["args"], **d["kw"], out=o, lse=lse, workspace=ws),
                rope=lambda: fm.rope(d["args"][0], None, f, q_out=o), write=lambda: fm.page_write(k, k, slots, *d["args"][1:5]),
                plan=lambda: fm.page_plan(**p))[name]
    call()
    torch.cuda.synchronize()
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]
    before = count()
    call()
    assert count() == before
