"""Workloads of the operators on a paged 8-bit K/V cache: the plan of a step
(block tables and slot maps from request lengths), rotary positions and their
gradient, the write of new keys and values into the pages, and the attention
over them.

Every case is run in one of two forms.  The plain form (``own`` false) is
elementary torch operations; the other makes the library calls a serving or
training program makes.  Both read the same inputs and return the same outputs.
"""
import math

import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
TOP = 448.0                      # e4m3's largest value
LOWEST, HIGHEST = -60, 60        # exponents of the scales that the write chooses


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a decode step of a small server: a token a request, few of which need a page
        dict(name="plan_decode", op="plan", B=64, S=4096, page=64, prompts=0, chunk=0, ended=2, ragged=True),
        # a large server: decodes, chunks of prompts, finished requests and taken-back drafts
        dict(name="plan_mixed", op="plan", B=700, S=8192, page=16, prompts=24, chunk=2000, ended=30, ragged=True),
        # queries and keys of a decode step at far positions: latency
        dict(name="rope_decode", op="rope", dtype="bf16", B=32, S=1, H=32, H_k=8, D=128, rot=128, layout="half", far=131072, grad=False),
        # a training batch
        dict(name="rope_train", op="rope", dtype="bf16", B=4, S=4096, H=32, H_k=8, D=128, rot=128, layout="half", far=0, grad=False),
        # its gradient where half of each head is rotated, by pairs of neighbours; odd length
        dict(name="rope_grad", op="rope", dtype="f16", B=8, S=2047, H=16, H_k=16, D=64, rot=32, layout="pairs", far=0, grad=True),
        # new keys and values of a decode step
        dict(name="write_decode", op="write", dtype="bf16", B=64, S=4096, H_k=8, page=64, new=1, ragged=True),
        # of prompts, into small pages
        dict(name="write_prompts", op="write", dtype="f16", B=5, S=4096, H_k=8, page=16, new=3333, ragged=True),
        # one user's next token after a chat-length context: latency
        dict(name="attn_single", op="attn", dtype="bf16", B=1, S=1000, H=32, H_k=8, page=64, new=1, ragged=False),
        # a served batch on ragged contexts
        dict(name="attn_decode", op="attn", dtype="bf16", B=64, S=8192, H=32, H_k=8, page=64, new=1, ragged=True),
        # long contexts in small pages, eight query heads a kv head, f16
        dict(name="attn_long", op="attn", dtype="f16", B=8, S=32768, H=64, H_k=8, page=16, new=1, ragged=True),
        # a few tokens a request: drafts that are checked, or the ends of prompts
        dict(name="attn_few", op="attn", dtype="bf16", B=16, S=6000, H=32, H_k=8, page=32, new=7, ragged=True),
        # chunks of prompts behind long contexts
        dict(name="attn_chunk", op="attn", dtype="bf16", B=4, S=8192, H=32, H_k=8, page=128, new=512, ragged=True),
    ]


_MOST_KEYS = 64 * 8192 * 8                 # cached keys x kv heads of the largest attention case
_MOST_PAIRS = 4 * 512 * 32 * 8192          # query heads x keys of the largest
_MOST_ROPE = 4 * 4096 * 40 * 128           # elements


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope", "write", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    H, H_k = rng.choice([(32, 8), (32, 8), (16, 16), (64, 8), (64, 4), (24, 8), (8, 1), (12, 4), (40, 8)])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "plan":
        B = _log(rng, 1, 700)
        return dict(op=op, B=B, S=_log(rng, 2, 8192), page=page, prompts=rng.randint(0, B // 3), chunk=_log(rng, 1, 2000),
                    ended=rng.randint(0, B // 3), ragged=rng.random() < 0.7)
    if op == "rope":
        hd = rng.choice([32, 64, 128, 128])
        S = _log(rng, 1, 8192)
        B = max(1, min(_log(rng, 1, 64), _MOST_ROPE // (S * (H + H_k) * hd)))
        return dict(op=op, dtype=dtype, B=B, S=S, H=H, H_k=H_k, D=hd, rot=hd if rng.random() < 0.5 else hd // 4 * rng.randint(1, 3),
                    layout=rng.choice(["half", "pairs"]), far=rng.choice([0, 0, 5000, 1 << 20]), grad=rng.random() < 0.4)
    B = _log(rng, 1, 128)
    if op == "write":
        S = _log(rng, 1, 8192)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, S)
        B = max(1, min(B, 5 * 3333 // new, 64 * 8192 // S))
        return dict(op=op, dtype=dtype, B=B, S=S, H_k=H_k, page=page, new=new, ragged=rng.random() < 0.7)
    S = _log(rng, 1, 65536)
    new = 1 if rng.random() < 0.5 else min(S, _log(rng, 1, 1024))
    S = max(new, min(S, _MOST_KEYS // (B * H_k), _MOST_PAIRS // (B * new * H)))
    B = max(1, min(B, _MOST_PAIRS // (S * new * H)))
    return dict(op=op, dtype=dtype, B=B, S=S, H=H, H_k=H_k, page=page, new=new, ragged=rng.random() < 0.7)


def _lengths(case):
    """Tokens of each sequence with the new ones, in no order: the case's
    length, or spread down to a quarter of it."""
    B, S, least = case["B"], case["S"], case.get("new", 1)
    if not case["ragged"]:
        return [S] * B
    return [max(min(S, least), S - (S * 3 // 4) * i // B) for i in range(B)]


def _news(case):
    """New tokens of each sequence."""
    n = case["new"]
    return [n - (i * 7) % max(1, n // 2) for i in range(case["B"])] if case["ragged"] else [n] * case["B"]


def _changes(case):
    """Cached tokens of each request and what the step does to them: a new
    token, a chunk of a prompt, the end (all tokens go), drafts taken back."""
    B, S = case["B"], case["S"]
    had = [max(1, S - (S * 3 // 4) * i // B) if case["ragged"] else S for i in range(B)]
    change = [1] * B
    for k in range(case["prompts"]):
        i = 3 * k % B
        had[i], change[i] = (had[i] // 2 if k % 2 else 0), case["chunk"] - (13 * k) % max(1, case["chunk"] // 2)
    for k in range(case["ended"]):
        i = (3 * k + 1) % B
        change[i] = -had[i] if k % 3 else -min(had[i], 5)
    return had, change


def _up(a, b):
    return (a + b - 1) // b


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _randn(shape, g, dtype, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    for part in x.view(-1).split(1 << 28):     # bounded fp32 temporaries
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(scale))
    return x


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _zeros(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def _table(held, width, page_ids, entry):
    """Block table [B, width]: held[b] pages of each sequence, in its entry's row; -1 elsewhere."""
    t = torch.full((len(held), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        t[entry[b], :n] = page_ids[at:at + n]
        at += n
    return t.cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    st = dict(case=case, op=case["op"])
    if case["op"] == "rope":
        B, S, H, H_k, hd = case["B"], case["S"], case["H"], case["H_k"], case["D"]
        dt = DTYPES[case["dtype"]]
        st["q"], st["k"] = _randn((B, S, H, hd), g, dt), _randn((B, S, H_k, hd), g, dt)
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=cpu)
        st["positions"] = (first + torch.arange(S)[None, :]).to(torch.int32).cuda() if case["far"] else None
        r = case["rot"]
        st["inv_freq"] = (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).cuda()
        st["magnitude"] = 1.0 if case["layout"] == "half" else 1.1386294361119891     # 0.1 ln 4 + 1: contexts four times as long
        st["q_out"], st["k_out"] = torch.zeros_like(st["q"]), torch.zeros_like(st["k"])
        return st
    B, page = case["B"], case["page"]
    entry = torch.randperm(B, generator=cpu)
    st["batch_idx"] = entry.to(torch.int32).cuda()                     # rows of the table in any order
    order = torch.randperm(B, generator=cpu).tolist()
    if case["op"] == "plan":
        had, change = _changes(case)
        had, change = [had[i] for i in order], [change[i] for i in order]
        held, width = [_up(x, page) for x in had], max(_up(max(x, x + n), page) for x, n in zip(had, change)) + 1
        taken = sum(max(0, _up(x + n, page) - _up(x, page)) for x, n in zip(had, change))
        spare = max(1, taken * 3 // 4)         # about as many as are given back, and at times too few
        ids = torch.randperm(sum(held) + spare, generator=cpu).to(torch.int32)
        st["table"] = _table(held, width, ids, entry)
        st["free_list"] = torch.full((len(ids),), -1, dtype=torch.int32, device="cuda")
        st["free_list"][:spare] = ids[sum(held):].cuda()
        st["n_free"], st["seqlen"], st["n_new"] = _int([spare]), _int(had), _int(change)
        st["rows"] = sum(max(0, n) for n in change) + 5                # as large as the program's buffers are
        st["slots"], st["positions"], st["cu_new"] = _zeros(st["rows"]), _zeros(st["rows"]), _zeros(B + 1)
        st["new_seqlen"], st["n_free_out"] = _zeros(B), _zeros(1)
        return st
    dt, H_k = DTYPES[case["dtype"]], case["H_k"]
    lens, news = _lengths(case), _news(case)
    lens = [lens[i] for i in order]
    held = [_up(x, page) for x in lens]
    n_pages = sum(held) + 3
    ids = torch.randperm(n_pages, generator=cpu).to(torch.int32)
    st["table"] = _table(held, max(held) + 1, ids, entry)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    N = cu[-1]
    for x in "kv":
        st[x + "_pages"] = _randn((n_pages, H_k, page, D), g, E4M3, 64.0)
        st[x + "_scale"] = torch.exp2(torch.randint(-8, -4, (n_pages, H_k), generator=g, device="cuda").float())
    if case["op"] == "write":
        st["k_new"], st["v_new"] = _randn((N, H_k, D), g, dt), _randn((N, H_k, D), g, dt)
        # heads of unequal size; now and then a token that its page's scale does not hold
        for x in ("k_new", "v_new"):
            st[x] *= torch.exp(torch.randn((1, H_k, 1), generator=g, device="cuda") +
                               3.0 * (torch.rand((N, 1, 1), generator=g, device="cuda") < 0.05)).to(dt)
        slots = []
        table = st["table"].cpu()
        for b in range(B):
            pos = torch.arange(lens[b] - news[b], lens[b])
            slots.append(table[entry[b], pos // page] * page + (pos % page).int())
        st["slots"] = torch.cat(slots).to(torch.int32).cuda()
        return st
    st["scale"] = D ** -0.5
    # queries of twice unit size: scores of a spread where few keys carry much of the weight
    st["q"] = _randn((N, case["H"], D), g, dt, 2.0)
    st["seqlen"], st["cu_q"], st["max_q"] = _int(lens), (_int(cu) if case["new"] > 1 else None), max(news)
    st["out"] = torch.zeros((N, case["H"], D), dtype=dt, device="cuda")
    st["lse"] = torch.zeros((N, case["H"]), dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"plan": _plain_plan, "rope": _plain_rope, "write": _plain_write, "attn": _plain_attn}[st["op"]](st)


def _run_own(st):
    from head_attention_forward_02_gb300 import fmha
    if st["op"] == "plan":
        fmha.page_plan(st["seqlen"], st["n_new"], st["table"], st["free_list"], st["n_free"], page_size=st["case"]["page"],
                       batch_idx=st["batch_idx"], slots=st["slots"], positions=st["positions"], cu_new=st["cu_new"],
                       new_seqlen=st["new_seqlen"], n_free_out=st["n_free_out"])
        return tuple(st[x] for x in ("table", "free_list", "n_free_out", "slots", "positions", "cu_new", "new_seqlen"))
    if st["op"] == "rope":
        f = fmha.rope_bwd if st["case"]["grad"] else fmha.rope
        return f(st["q"], st["k"], st["inv_freq"], positions=st["positions"], interleaved=st["case"]["layout"] == "pairs",
                 magnitude=st["magnitude"], q_out=st["q_out"], k_out=st["k_out"])
    pool = (st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"])
    if st["op"] == "write":
        fmha.page_write(st["k_new"], st["v_new"], st["slots"], *pool)
        return pool
    return fmha.page_fwd(st["q"], *pool, st["table"], st["seqlen"], cu_q=st["cu_q"], max_q=st["max_q"],
                         batch_idx=st["batch_idx"], scale=st["scale"], out=st["out"], lse=st["lse"])


def _plain_plan(st):
    page, e = st["case"]["page"], st["batch_idx"].long()
    L, n, table, free = st["seqlen"].long(), st["n_new"].long(), st["table"], st["free_list"]
    dev, width, spare = L.device, st["table"].shape[1], st["n_free"].long()
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    after = torch.maximum(L + n, zero)
    had, want = (L + page - 1) // page, (after + page - 1) // page
    # pages that become empty, in order, onto the stack
    i = torch.arange(width, device=dev)[None, :]
    gone = (i >= want[:, None]) & (i < had[:, None])
    given = gone.sum(1)
    at = spare + (torch.cumsum(given, 0) - given)[:, None] + i - want[:, None]
    rows = table.long()[e]
    stack = torch.cat([free.long(), zero])                             # the last element takes what is not given
    stack[torch.where(gone, at, len(free))] = rows
    stack = stack[:-1]
    # pages from its top, for the requests that all fit
    total = spare + given.sum()
    need = torch.maximum(want - had, zero)
    c = torch.cumsum(need, 0)
    ok = (need == 0) | (c <= total)
    new = (i >= had[:, None]) & (i < want[:, None]) & ok[:, None]
    src = total - 1 - ((c - need)[:, None] + i - had[:, None])
    rows = torch.where(new, stack[src.clamp(0, len(free) - 1)], rows)
    table[e] = rows.to(torch.int32)
    left = total - torch.where(ok & (need > 0), c, 0).max()
    kept = torch.where(n < 0, after, torch.where(ok, L + n, L))
    # the tokens' positions and slots
    count = torch.maximum(n, zero)
    cu = torch.cat([zero, torch.cumsum(count, 0)])
    t = torch.arange(st["rows"], device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=len(L) - 1)
    real = t < cu[-1]
    pos = L[b] + t - cu[b]
    slot = rows[b, (pos // page).clamp(0, width - 1)] * page + pos % page
    slot = torch.where(real & ok[b], slot, -1)
    free.copy_(stack)
    return (table, free, left.to(torch.int32), slot.to(torch.int32), torch.where(real, pos, -1).to(torch.int32),
            cu.to(torch.int32), kept.to(torch.int32))


def _plain_rope(st):
    c, dt = st["case"], st["q"].dtype
    r = c["rot"]
    pos = st["positions"] if st["positions"] is not None else torch.arange(c["S"], device="cuda")[None, :].expand(c["B"], c["S"])
    angle = pos.double()[..., None] * st["inv_freq"]                    # far positions: 64 bits
    cos = (torch.cos(angle) * st["magnitude"]).float()[:, :, None]
    sin = (torch.sin(angle) * st["magnitude"]).float()[:, :, None]
    if c["grad"]:
        sin = -sin
    def turn(x):
        x = x.float()
        if c["layout"] == "half":
            a, b = x[..., :r // 2], x[..., r // 2:r]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([y, x[..., r:]], -1).to(dt)
    return turn(st["q"]), turn(st["k"])


def _plain_write(st):
    page, slots = st["case"]["page"], st["slots"].long()
    n_pages, H_k = st["k_scale"].shape
    p, off = slots // page, slots % page
    first = torch.full((n_pages,), page, dtype=torch.int64, device=p.device).scatter_reduce(0, p, off, "amin")   # first new row of a page
    j = torch.arange(page, device=p.device)[None, None, :, None]
    for x in "kv":
        new, pages, scale = st[x + "_new"].float(), st[x + "_pages"], st[x + "_scale"]
        top = torch.zeros((n_pages, H_k), device=p.device).scatter_reduce(
            0, p[:, None].expand(-1, H_k), new.abs().amax(-1), "amax")
        m, ex = torch.frexp(top / TOP)                                  # top / 448 = m 2^ex, m in [1/2, 1)
        ex = torch.where(m == 0.5, ex - 1, ex).clamp(LOWEST, HIGHEST)
        ex = torch.where(top > 0, ex, LOWEST)
        was = torch.where(first[:, None] > 0, scale, 0.0)
        now = torch.where(first[:, None] < page, torch.maximum(was, torch.ldexp(torch.ones_like(top), ex)), scale)
        # rows before the first new one, where the scale grew
        old = (j < first[:, None, None, None]) & (now > scale)[:, :, None, None]
        codes = pages.view(torch.uint8)
        again = (pages.float() * (scale / now)[:, :, None, None]).to(E4M3).view(torch.uint8)
        codes.copy_(torch.where(old, again, codes))
        y = (new / now[p][..., None]).clamp(-TOP, TOP).to(E4M3).view(torch.uint8)
        codes[p, :, off] = y
        scale.copy_(now)
    return st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"]


def _gathered(st, x):
    """Keys or values of each sequence in order, fp32: [B, H_k, tokens, D]."""
    pages, scale = st[x + "_pages"], st[x + "_scale"]
    t = st["table"].long()[st["batch_idx"].long()].clamp(min=0)
    y = pages.view(torch.uint8)[t].view(E4M3).float() * scale[t][..., None, None]
    return y.permute(0, 2, 1, 3, 4).reshape(t.shape[0], pages.shape[1], -1, D)


def _plain_attn(st):
    q, L, c = st["q"], st["seqlen"].long(), st["case"]
    (N, H, _), H_k, B, n_max = q.shape, c["H_k"], c["B"], st["max_q"]
    G, dev = H // H_k, q.device
    cu = st["cu_q"].long() if st["cu_q"] is not None else torch.arange(B + 1, device=dev)
    n = cu[1:] - cu[:-1]
    t = torch.arange(n_max, device=dev)
    row = (cu[:-1, None] + t).clamp(max=N - 1)                          # [B, n_max]: rows past a sequence's own are dropped below
    k, v = _gathered(st, "k"), _gathered(st, "v")
    S = k.shape[2]
    qf = (q.float() * st["scale"])[row].view(B, n_max, H_k, G, D).permute(0, 2, 1, 3, 4).reshape(B, H_k, n_max * G, D)
    s = qf @ k.transpose(2, 3)
    seen = torch.arange(S, device=dev) <= (L - n)[:, None, None] + t[None, :, None]      # [B, n_max, S]
    seen = (seen & (torch.arange(S, device=dev) < L[:, None, None])).repeat_interleave(G, dim=1)[:, None]
    s = s.masked_fill_(~seen, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s.sub_(torch.where(m == -math.inf, 0.0, m)))
    l = p.sum(dim=-1, keepdim=True)
    o = torch.where(l > 0, (p @ v) / l, 0.0)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)
    o = o.view(B, H_k, n_max, G, D).permute(0, 2, 1, 3, 4).reshape(B, n_max, H, D)
    lse = lse.view(B, H_k, n_max, G).permute(0, 2, 1, 3).reshape(B, n_max, H)
    i = torch.arange(N, device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    return o[b, i - cu[b]].to(q.dtype), lse[b, i - cu[b]]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "plan":
        had, change = _changes(case)
        page = case["page"]
        moved = sum(abs(_up(x + n, page) - _up(x, page)) for x, n in zip(had, change))
        tokens = sum(max(0, n) for n in change)
        touched = sum(_up(x + n, page) - x // page for x, n in zip(had, change) if n > 0)   # table entries read for slots
        return {"bytes": 20 * case["B"] + 8 * moved + 8 * tokens + 4 * touched, "flops": 0}
    if case["op"] == "rope":
        x = case["B"] * case["S"] * (case["H"] + case["H_k"])
        return {"bytes": 4 * x * case["D"] + 4 * case["rot"] + (4 * case["B"] * case["S"] if case["far"] else 0),
                "flops": 3 * x * case["rot"]}
    lens, news, H_k, page = _lengths(case), _news(case), case["H_k"], case["page"]
    if case["op"] == "write":
        pages = sum(_up(L, page) - (L - n) // page for L, n in zip(lens, news))
        return {"bytes": sum(news) * (H_k * D * 6 + 4) + 16 * pages * H_k, "flops": 0}
    H = case["H"]
    pairs = sum(n * L - n * (n - 1) // 2 for L, n in zip(lens, news))
    pages = sum(_up(L, page) for L in lens)
    return {"bytes": 2 * D * H_k * sum(lens) + pages * (8 * H_k + 4) + sum(news) * H * (4 * D + 4) + 8 * case["B"],
            "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None                                                     # whole numbers
    st = prepare(case, seed)
    if case["op"] == "rope":
        r, B, S = case["rot"], case["B"], case["S"]
        outs = []
        for x in (st["q"], st["k"]):
            y = x.double()
            for b in range(B):
                pos = st["positions"][b].double() if st["positions"] is not None else torch.arange(S, device="cuda").double()
                # a rotation as a product with a complex number of size `magnitude`
                z = torch.polar(torch.full((S, r // 2), st["magnitude"], dtype=torch.float64, device="cuda"),
                                torch.outer(pos, st["inv_freq"]) * (-1.0 if case["grad"] else 1.0))[:, None]
                first, second = (slice(0, r // 2), slice(r // 2, r)) if case["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
                w = torch.complex(y[b, :, :, first], y[b, :, :, second]) * z
                y[b, :, :, first], y[b, :, :, second] = w.real, w.imag
            outs.append(y)
        return tuple(outs)
    page, H_k = case["page"], case["H_k"]
    if case["op"] == "write":
        outs = []
        slots = st["slots"].cpu().tolist()
        runs = {}
        for i, s in enumerate(slots):                                   # page: its first new token, row and count
            if s // page in runs:
                runs[s // page][2] += 1
            else:
                runs[s // page] = [i, s % page, 1]
        for x in "kv":
            pages, scale, new = st[x + "_pages"].float().double(), st[x + "_scale"].double(), st[x + "_new"].double()
            tops = {p: new[i:i + n].abs().amax((0, 2)) for p, (i, _, n) in runs.items()}
            for p, (i, row, n) in runs.items():
                # the smallest power of two that brings the largest value to 448 or less
                e = torch.ceil(torch.log2(tops[p] / TOP) - 1e-12).clamp(LOWEST, HIGHEST)
                s = torch.pow(2.0, e)
                if row > 0:
                    s = torch.maximum(s, scale[p])
                    pages[p, :, :row] *= (scale[p] / s)[:, None, None]
                pages[p, :, row:row + n] = (new[i:i + n] / s[None, :, None]).transpose(0, 1)
                scale[p] = s
            outs.append((pages, scale))
        return outs[0][0], outs[1][0], outs[0][1], outs[1][1]
    H, B = case["H"], case["B"]
    G = H // H_k
    o, lse = st["out"].double(), st["lse"].double()
    cu = st["cu_q"].tolist() if st["cu_q"] is not None else list(range(B + 1))
    for b in range(B):
        L, n = int(st["seqlen"][b]), cu[b + 1] - cu[b]
        ids = st["table"][int(st["batch_idx"][b]), :_up(L, page)].long()
        keys, vals = ((st[x + "_pages"].view(torch.uint8)[ids].view(E4M3).float().double() *
                       st[x + "_scale"][ids].double()[:, :, None, None]).transpose(0, 1).reshape(H_k, -1, D)[:, :L] for x in "kv")
        hide = torch.ones((n, L), dtype=torch.bool, device="cuda").triu(L - n + 1)
        for g in range(H_k):
            x = torch.einsum("thd,kd->htk", st["q"][cu[b]:cu[b + 1], g * G:(g + 1) * G].double(), keys[g]) * st["scale"]
            x = x.masked_fill(hide, -math.inf)
            z = torch.logsumexp(x, dim=-1)
            o[cu[b]:cu[b + 1], g * G:(g + 1) * G] = torch.einsum("htk,kd->thd", torch.exp(x - z[..., None]), vals[g])
            lse[cu[b]:cu[b + 1], g * G:(g + 1) * G] = z.T
    return o, lse
