"""Workloads of the cache operators: attention of drafted token trees over a
K/V cache, the commit of the accepted drafts, the accumulation of attention
weight per cached key, and the eviction of the keys with the least of it.

Every case is run in one of two forms.  The plain form (``own`` false) is
elementary torch operations in fp32; the other makes the library calls a
serving program makes.  Both read the same inputs and return the same outputs.
"""
import math

import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
ESIZE = {"bf16": 2, "f16": 2, "e4m3": 1}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user, a short draft after a chat-length context: latency
        dict(name="tree_single", op="tree", dtype="bf16", B=1, T=8, H=32, H_k=8, S=1000, ragged=False, chain=False),
        # a served batch with ragged contexts and drafts of unequal size
        dict(name="tree_batch", op="tree", dtype="f16", B=16, T=27, H=32, H_k=8, S=4096, ragged=True, chain=False),
        # a full batch on long contexts with wide trees: two 128-row query blocks a kv head
        dict(name="tree_large", op="tree", dtype="bf16", B=32, T=64, H=32, H_k=8, S=8192, ragged=False, chain=False),
        # an fp8 cache, few kv heads, long ragged contexts and a linear draft
        dict(name="tree_fp8", op="tree", dtype="e4m3", B=16, T=5, H=64, H_k=8, S=16384, ragged=True, chain=True),
        # accept a draft of one user / of a large batch with wide trees
        dict(name="commit_single", op="commit", dtype="bf16", B=1, T=8, H=32, H_k=8, S=1000, ragged=False),
        dict(name="commit_batch", op="commit", dtype="bf16", B=64, T=64, H=32, H_k=8, S=2048, ragged=True),
        # weights of one generated token a sequence, every step of a decode loop
        dict(name="weights_decode", op="weights", dtype="bf16", B=32, Sq=1, H=32, H_k=8, S=8192, ragged=True, mask="none"),
        # weights of the last queries of a long prompt (an observation window)
        dict(name="weights_window", op="weights", dtype="e4m3", B=4, Sq=33, H=64, H_k=8, S=16384, ragged=True, mask="causal"),
        # weights of every query of a prompt
        dict(name="weights_prompt", op="weights", dtype="bf16", B=1, Sq=4096, H=32, H_k=8, S=4096, ragged=False, mask="causal"),
        # one sequence just over its budget: latency
        dict(name="evict_single", op="evict", dtype="bf16", B=1, H=32, H_k=8, S=1300, S_out=1024, budget=1000, recent=100, ragged=False),
        # a batch of long prompts into the decode cache
        dict(name="evict_batch", op="evict", dtype="bf16", B=32, H=32, H_k=8, S=8192, S_out=2304, budget=2048, recent=256, ragged=True),
        # few long fp8 contexts, a small budget: the selection reads more than the move
        dict(name="evict_long", op="evict", dtype="e4m3", B=2, H=64, H_k=8, S=65536, S_out=4096, budget=2047, recent=65, ragged=False),
    ]


_LARGEST_PAIRS = 32 * 64 * 32 * 8192       # query heads x keys of the largest tree case
_LARGEST_KEYS = 32 * 8192 * 8              # cached keys x kv heads


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "commit", "weights", "weights", "evict"])
    H, H_k = rng.choice([(32, 8), (32, 8), (16, 16), (64, 8), (64, 2), (24, 8), (8, 1), (12, 4)])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "e4m3"]), H=H, H_k=H_k, ragged=rng.random() < 0.6)
    B = _log(rng, 1, 32)
    if op == "tree":
        T = _log(rng, 1, 64)
        S = _log(rng, 1, 32768)
        S = min(S, _LARGEST_KEYS // (B * H_k), _LARGEST_PAIRS // (B * T * H))
        c.update(B=B, T=T, S=max(1, S), chain=rng.random() < 0.3)
    elif op == "commit":
        T = _log(rng, 1, 64)
        S = max(T, _log(rng, 1, 8192))
        c.update(B=B, T=T, S=S)
    elif op == "weights":
        if rng.random() < 0.3:
            S = _log(rng, 128, 4096)
            c.update(B=min(B, max(1, 4096 * 4096 // (S * S))), Sq=S, S=S, mask="causal", ragged=False)
            if c["H"] > 32:
                c.update(H=32, H_k=4)
        else:
            Sq = _log(rng, 1, 128)
            S = max(Sq, _log(rng, 1, 32768))
            S = max(Sq, min(S, _LARGEST_KEYS // (B * H_k), 4096 * 4096 * 32 // (B * Sq * H)))
            c.update(B=B, Sq=Sq, S=S, mask=rng.choice(["none", "causal"]))
    else:
        S = min(_log(rng, 2, 65536), _LARGEST_KEYS // (B * H_k))
        budget = _log(rng, 1, max(1, min(S, 4096)))
        c.update(B=B, S=S, budget=budget, recent=rng.randint(0, budget), S_out=budget + rng.randint(0, 256))
    return c


def _lengths(case):
    """Cached tokens of each sequence, in no order: the case's full length, or
    spread down to a quarter of it."""
    B, S = case["B"], case["S"]
    room = case["T"] if case["op"] == "commit" else 0
    least = min(S, case["Sq"]) if case["op"] == "weights" and case["mask"] == "causal" else 0
    hi = S - room
    if not case["ragged"]:
        return [hi] * B
    return [max(least, hi - (hi * 3 // 4) * i // B) for i in range(B)]


def _counts(n, B, ragged):
    """Valid tokens of each sequence of a padded batch."""
    return [n - (i * 7) % max(1, n // 2) for i in range(B)] if ragged else [n] * B


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


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    op, B, S, H, H_k = case["op"], case["B"], case["S"], case["H"], case["H_k"]
    dt = DTYPES[case["dtype"]]
    lens = _lengths(case)
    lens = [lens[i] for i in torch.randperm(B, generator=cpu).tolist()]
    st = dict(case=case, op=op, scale=D ** -0.5, seqlen=_int(lens))
    st["batch_idx"] = torch.randperm(B, generator=cpu).to(torch.int32).cuda()   # cache entries in any order
    st["k_cache"] = _randn((B, S, H_k, D), g, dt)
    if op != "weights":
        st["v_cache"] = _randn((B, S, H_k, D), g, dt)
    if op in ("tree", "commit"):
        T = case["T"]
        st["k_new"] = _randn((B, T, H_k, D), g, dt)
        st["v_new"] = _randn((B, T, H_k, D), g, dt)
    if op == "tree":
        # queries of twice unit size: scores of a spread where few keys carry much of the weight
        st["q"] = _randn((B, T, H, D), g, dt, 2.0)
        st["n_draft"] = _int(_counts(T, B, case["ragged"]))
        st["tree_mask"] = None if case["chain"] else _tree_masks(B, T, cpu).cuda()
        st["out"] = torch.zeros((B, T, H, D), dtype=dt, device="cuda")
        st["lse"] = torch.zeros((B, H, T), dtype=torch.float32, device="cuda")
    elif op == "commit":
        st["path"], st["n_accept"] = _paths(B, T, cpu)
    elif op == "weights":
        Sq = case["Sq"]
        st["q"] = _randn((B, Sq, H, D), g, dt, 2.0)
        st["n_query"] = _int([min(n, L) if case["mask"] == "causal" else n
                              for n, L in zip(_counts(Sq, B, case["ragged"]), lens)])
        # the log-sum-exp that the attention call before this one returned
        s = _scores(st["q"], _entries(st, "k_cache"), st["scale"], H_k).masked_fill_(~_weights_visible(st), -math.inf)
        st["lse"] = torch.logsumexp(s, dim=-1).view(B, H_k, Sq, H // H_k).permute(0, 1, 3, 2).reshape(B, H, Sq).contiguous()
        del s
        st["acc"] = torch.rand((B, H_k, S), generator=g, device="cuda") * 0.01
        st["out"] = torch.zeros((B, H_k, S), dtype=torch.float32, device="cuda")
    else:
        # accumulated weights: a heavy tail, and many keys that never got any
        a = torch.exp(2.0 * torch.randn((B, H_k, S), generator=g, device="cuda")) / S
        st["acc"] = torch.where(torch.rand((B, H_k, S), generator=g, device="cuda") < 0.2, torch.zeros_like(a), a)
        So = case["S_out"]
        st["k_out"] = torch.zeros((B, So, H_k, D), dtype=dt, device="cuda")
        st["v_out"] = torch.zeros((B, So, H_k, D), dtype=dt, device="cuda")
        st["acc_out"] = torch.zeros((B, H_k, So), dtype=torch.float32, device="cuda")
        st["kept"] = torch.zeros((B, H_k, case["budget"]), dtype=torch.int32, device="cuda")
        st["new_seqlen"] = torch.zeros((B,), dtype=torch.int32, device="cuda")
    return st


def _tree_masks(B, T, cpu):
    """Ancestor masks of random trees: draft i descends from a draft before it,
    or from the last cached token."""
    m = torch.zeros((B, T, T), dtype=torch.bool)
    parent = (torch.rand((B, T), generator=cpu) * (torch.arange(T) + 1)).long() - 1      # -1 .. i - 1
    for i in range(T):
        has = parent[:, i] >= 0
        m[:, i] = m[torch.arange(B), parent[:, i].clamp(min=0)] & has[:, None]
        m[:, i, i] = True
    return m


def _paths(B, T, cpu):
    """Accepted drafts of each sequence, in order, and how many."""
    n = torch.randint(1, T + 1, (B,), generator=cpu)
    path = torch.full((B, T), -1, dtype=torch.int64)
    for b in range(B):
        k = int(n[b])
        path[b, :k] = torch.randperm(T, generator=cpu)[:k].sort().values
    return path.to(torch.int32).cuda(), n.to(torch.int32).cuda()


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"tree": _plain_tree, "commit": _plain_commit, "weights": _plain_weights, "evict": _plain_evict}[st["op"]](st)


def _run_own(st):
    from head_attention_forward_02_gb300 import fmha
    if st["op"] == "tree":
        return fmha.tree_fwd(st["q"], st["k_cache"], st["v_cache"], st["k_new"], st["v_new"], st["seqlen"],
                             tree_mask=st["tree_mask"], n_draft=st["n_draft"], batch_idx=st["batch_idx"],
                             scale=st["scale"], out=st["out"], lse=st["lse"])
    if st["op"] == "commit":
        fmha.tree_commit(st["k_cache"], st["v_cache"], st["k_new"], st["v_new"], st["seqlen"], st["path"],
                         st["n_accept"], batch_idx=st["batch_idx"])
        return st["k_cache"], st["v_cache"]
    if st["op"] == "weights":
        return fmha.cache_weights(st["q"], st["k_cache"], st["lse"], st["seqlen"], acc=st["acc"], out=st["out"],
                                  n_query=st["n_query"], batch_idx=st["batch_idx"], mask=st["case"]["mask"],
                                  scale=st["scale"])
    fmha.cache_evict(st["k_cache"], st["v_cache"], st["acc"], st["seqlen"], st["case"]["budget"],
                     recent=st["case"]["recent"], batch_idx=st["batch_idx"], k_out=st["k_out"], v_out=st["v_out"],
                     acc_out=st["acc_out"], kept=st["kept"], new_seqlen=st["new_seqlen"])
    return st["k_out"], st["v_out"], st["acc_out"], st["kept"], st["new_seqlen"]


def _entries(st, name):
    """Each sequence's entry of a cache, in sequence order."""
    return st[name].view(torch.uint8)[st["batch_idx"].long()].view(st[name].dtype) if st[name].element_size() == 1 \
        else st[name][st["batch_idx"].long()]


def _scores(q, k, scale, H_k):
    """fp32 scores [B, H_k, T * G, keys] of q [B, T, H, D] on k [B, keys, H_k, D]; row t * G + i is head i of the group."""
    B, T, H, _ = q.shape
    qf = q.float().view(B, T, H_k, H // H_k, D).permute(0, 2, 1, 3, 4).reshape(B, H_k, -1, D)
    return (qf * scale) @ k.float().permute(0, 2, 3, 1)


def _plain_tree(st):
    q, H_k = st["q"], st["case"]["H_k"]
    B, T, H, _ = q.shape
    G, S, dev = H // H_k, st["case"]["S"], q.device
    k, v = _entries(st, "k_cache"), _entries(st, "v_cache")
    s = torch.cat([_scores(q, k, st["scale"], H_k), _scores(q, st["k_new"], st["scale"], H_k)], dim=-1)
    cached = torch.arange(S, device=dev)[None, :] < st["seqlen"][:, None]                      # [B, S]
    draft = torch.arange(T, device=dev)[None, :] < st["n_draft"][:, None]                      # [B, T]
    tree = st["tree_mask"] if st["tree_mask"] is not None else \
        torch.ones((T, T), dtype=torch.bool, device=dev).tril().expand(B, T, T)
    seen = torch.cat([cached[:, None, :].expand(B, T, S), tree & draft[:, None, :]], dim=-1)   # [B, T, S + T]
    s = s.masked_fill_(~seen.repeat_interleave(G, dim=1)[:, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s.sub_(torch.where(m == -math.inf, 0.0, m)))
    l = p.sum(dim=-1, keepdim=True)
    o = p[..., :S] @ v.float().permute(0, 2, 1, 3) + p[..., S:] @ st["v_new"].float().permute(0, 2, 1, 3)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    o = o.view(B, H_k, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, H, D)
    lse = lse.view(B, H_k, T, G).permute(0, 1, 3, 2).reshape(B, H, T)
    # rows past a sequence's drafts stay as they are
    o = torch.where(draft[:, :, None, None], o, st["out"].float()).to(q.dtype)
    return o, torch.where(draft[:, None, :], lse, st["lse"])


def _plain_commit(st):
    B, T = st["path"].shape
    i = torch.arange(T, device=st["path"].device)[None, :]
    b = torch.arange(B, device=st["path"].device)[:, None]
    accepted = (i < st["n_accept"][:, None])[..., None, None]
    draft = st["path"].long().clamp(min=0)
    entry, row = st["batch_idx"].long()[:, None], st["seqlen"].long()[:, None] + i
    for cache, new in ((st["k_cache"], st["k_new"]), (st["v_cache"], st["v_new"])):
        bits = {1: torch.uint8, 2: torch.int16}[cache.element_size()]
        cache, new = cache.view(bits), new.view(bits)
        cache[entry, row] = torch.where(accepted, new[b, draft], cache[entry, row])     # others keep their rows
    return st["k_cache"], st["v_cache"]


def _weights_visible(st):
    """[B, 1, Sq * G, S]: whether a query sees a cached key."""
    q, dev = st["q"], st["q"].device
    B, Sq, H, _ = q.shape
    G, S = H // st["case"]["H_k"], st["case"]["S"]
    j = torch.arange(S, device=dev)[None, None, :]
    i = torch.arange(Sq, device=dev)[None, :, None]
    n, L = st["n_query"][:, None, None], st["seqlen"][:, None, None]
    seen = (j < L) & (i < n)
    if st["case"]["mask"] == "causal":
        seen = seen & (j <= i + L - n)
    return seen.repeat_interleave(G, dim=1)[:, None]


def _plain_weights(st):
    q, H_k = st["q"], st["case"]["H_k"]
    B, Sq, H, _ = q.shape
    G, S = H // H_k, st["case"]["S"]
    s = _scores(q, _entries(st, "k_cache"), st["scale"], H_k)
    lse = st["lse"].view(B, H_k, G, Sq).permute(0, 1, 3, 2).reshape(B, H_k, Sq * G, 1)
    lse = torch.where(lse == -math.inf, torch.zeros_like(lse), lse)                            # a row without keys
    w = torch.exp(s.sub_(lse)).masked_fill_(~_weights_visible(st), 0.0).sum(dim=2)             # [B, H_k, S]
    e = st["batch_idx"].long()
    new = st["acc"][e] + w
    cached = torch.arange(S, device=q.device)[None, None, :] < st["seqlen"][:, None, None]
    out = st["out"].clone()
    out[e] = torch.where(cached, new, out[e])
    return out


def _plain_evict(st):
    c, e = st["case"], st["batch_idx"].long()
    B, H_k, S, budget, So = c["B"], c["H_k"], c["S"], c["budget"], c["S_out"]
    dev = e.device
    j = torch.arange(S, device=dev)[None, None, :]
    L = st["seqlen"][:, None, None]
    acc = st["acc"][e]
    score = torch.where(j < L, torch.where(j >= L - c["recent"], math.inf, acc.double()), -math.inf)
    new_len = st["seqlen"].clamp(max=budget)
    first = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :budget]
    i = torch.arange(budget, device=dev)[None, None, :]
    has = i < new_len[:, None, None]
    first = torch.cat([first, first.new_full((B, H_k, budget - first.shape[-1]), S)], -1) if first.shape[-1] < budget else first
    kept = torch.sort(torch.where(has, first, S), dim=-1).values
    src = kept.clamp(max=S - 1)
    has = has.expand(B, H_k, budget)
    acc_out = torch.zeros((B, H_k, So), dtype=torch.float32, device=dev)
    acc_out[..., :budget] = torch.where(has, acc.gather(2, src), 0.0)
    outs = []
    for cache, was in ((st["k_cache"], st["k_out"]), (st["v_cache"], st["v_out"])):
        bits = {1: torch.uint8, 2: torch.int16}[cache.element_size()]
        rows = cache.view(bits)[e[:, None, None], src, torch.arange(H_k, device=dev)[None, :, None]]   # [B, H_k, budget, D]
        out = was.clone()
        out.view(bits)[:, :budget] = torch.where(has[..., None], rows, was.view(bits)[:, :budget].transpose(1, 2)).transpose(1, 2)
        outs.append(out)
    return outs[0], outs[1], acc_out, torch.where(has, kept, -1).to(torch.int32), new_len.to(torch.int32)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, B, H, H_k, E = case["op"], case["B"], case["H"], case["H_k"], ESIZE[case["dtype"]]
    lens, row = _lengths(case), H_k * D * E               # one token's keys (or values)
    if op == "tree":
        n = _counts(case["T"], B, case["ragged"])
        seen = sum(x * L + x * (x + 1) // 2 for x, L in zip(n, lens))        # at most: a chain sees every draft before it
        return {"bytes": 2 * row * (sum(lens) + sum(n)) + sum(n) * H * (2 * D * E + 4)
                + (0 if case["chain"] else sum(x * x for x in n)) + 12 * B,
                "flops": 4 * D * H * seen}
    if op == "commit":
        accepted = B * (case["T"] + 1) / 2                # on average
        return {"bytes": 4 * row * accepted + 4 * accepted + 12 * B, "flops": 0}
    if op == "weights":
        n = [min(x, L) if case["mask"] == "causal" else x for x, L in zip(_counts(case["Sq"], B, case["ragged"]), lens)]
        seen = sum(x * L - (x * (x - 1) // 2 if case["mask"] == "causal" else 0) for x, L in zip(n, lens))
        return {"bytes": row * sum(lens) + sum(n) * H * (D * E + 4) + 8 * H_k * sum(lens) + 12 * B,
                "flops": 2 * D * H * seen}
    kept = sum(min(L, case["budget"]) for L in lens)
    return {"bytes": 4 * row * kept + 4 * H_k * sum(lens) + 4 * H_k * (B * case["S_out"] + B * case["budget"]) + 12 * B,
            "flops": 0}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] not in ("tree", "weights"):
        return None                                       # bits that are moved, whole numbers
    st = prepare(case, seed)
    B, H, H_k, S = case["B"], case["H"], case["H_k"], case["S"]
    G = H // H_k
    if case["op"] == "tree":
        o, lse = st["out"].double(), st["lse"].double()
        for b in range(B):
            L, n, e = int(st["seqlen"][b]), int(st["n_draft"][b]), int(st["batch_idx"][b])
            tree = st["tree_mask"][b, :n, :n].bool() if st["tree_mask"] is not None else \
                torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
            see = torch.cat([torch.ones((n, L), dtype=torch.bool, device="cuda"), tree], 1)
            for g in range(H_k):
                keys = torch.cat([st["k_cache"][e, :L, g].double(), st["k_new"][b, :n, g].double()])
                vals = torch.cat([st["v_cache"][e, :L, g].double(), st["v_new"][b, :n, g].double()])
                x = torch.einsum("thd,kd->htk", st["q"][b, :n, g * G:(g + 1) * G].double(), keys) * st["scale"]
                x = x.masked_fill(~see, -math.inf)
                z = torch.logsumexp(x, dim=-1)
                w = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[..., None])
                o[b, :n, g * G:(g + 1) * G] = torch.einsum("htk,kd->thd", w, vals)
                lse[b, g * G:(g + 1) * G, :n] = z
        return o, lse
    out = st["out"].double()
    for b in range(B):
        L, n, e = int(st["seqlen"][b]), int(st["n_query"][b]), int(st["batch_idx"][b])
        for h in range(H):
            g = h // G
            if h % G == 0:
                out[e, g, :L] = st["acc"][e, g, :L].double()
            x = st["q"][b, :n, h].double() @ st["k_cache"][e, :L, g].double().T * st["scale"]
            w = torch.exp(x - st["lse"][b, h, :n].double()[:, None])
            if case["mask"] == "causal":
                w = torch.tril(w, diagonal=L - n)
            out[e, g, :L] += w.sum(dim=0)
    return out
