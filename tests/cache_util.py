"""Plain 64-bit forms of the cache operators (drafted trees, weight
accumulation), their inputs, and the error bounds the GPU tests hold them to."""
from __future__ import annotations

import math

import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
# half a rounding step (relative), smallest normal, half the subnormal step
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4}
NORMAL = {"bf16": 2.0 ** -126, "f16": 2.0 ** -14, "e4m3": 2.0 ** -6}
SUBHALF = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10}
SENTINEL = 0x3C


def draw(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(DTYPES[dtype])


def f64(t):
    return t.double() if t.element_size() > 1 else t.float().double()


def sentinel(shape, dtype, device="cuda"):
    """A tensor of a known bit pattern: what a call must leave alone keeps it."""
    n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
    return torch.full((n,), SENTINEL, dtype=torch.uint8, device=device).view(dtype).view(shape)


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == SENTINEL).all()) if t.numel() else True


def fill_nan(t, index):
    """NaN in t[index]: all ones is a NaN of e4m3, fp16 and bf16 alike."""
    t.view(torch.uint8).view(*t.shape, t.element_size())[index] = 0xFF


def take(t, rows):
    """t[rows] of rows of any type (torch does not index e4m3 on the CPU)."""
    return t.contiguous().view(torch.uint8)[rows].view(t.dtype)


def random_tree(gen, B, T):
    """Ancestor masks of random trees over T drafts (draft i's parent is before it, or the cache)."""
    m = torch.zeros((B, T, T), dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            p = int(torch.randint(-1, i, (1,), generator=gen)) if i else -1
            if p >= 0:
                m[b, i] = m[b, p]
            m[b, i, i] = True
    return m


def attend(q, keys, vals, see, scale, out_scale, dtype):
    """One sequence and kv head: q [n, G, D], keys / vals [K, D], see [n, K].
    Returns O [n, G, D], LSE [n, G] and the bounds on their errors."""
    n, G, _ = q.shape
    x = torch.einsum("tgd,kd->tgk", q, keys) * scale
    a = (torch.einsum("tgd,kd->tgk", q.abs(), keys.abs()) * scale).amax(-1) if keys.shape[0] else torch.zeros(n, G).double()
    x = x.masked_fill(~see[:, None, :], -math.inf)
    lse = torch.logsumexp(x, -1) if keys.shape[0] else torch.full((n, G), -math.inf).double()
    empty = lse == -math.inf
    w = torch.exp(x - torch.where(empty, 0.0, lse)[..., None])
    o = torch.einsum("tgk,kd->tgd", w, vals) * out_scale
    # a score is a sum of 128 products in fp32, each addition off by at most
    # 2^-23 of the partial sum (bounded by a); the exponential of its scaled
    # value, and the row sum and the joins, a few fp32 roundings more
    ds = a * 130 * 2.0 ** -23 + lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -21 + 1e-5
    wabs = torch.einsum("tgk,kd->tgd", w, vals.abs()) * abs(out_scale)
    # weights are rounded to the type relative to a reference that leaves the
    # largest at 1 or more, so an underflowing one is off by at most SUBHALF of the largest
    wmax = w.amax(-1, keepdim=True) if keys.shape[0] else torch.zeros(n, G, 1).double()
    low = torch.einsum("tgk,kd->tgd", (w < NORMAL[dtype] * wmax).double(), vals.abs()) * abs(out_scale)
    tol = wabs * (HALF[dtype] + 2 * ds[..., None]) + SUBHALF[dtype] * wmax * low
    tol = tol + (o.abs() + tol) * HALF[dtype] + SUBHALF[dtype]                # O's own rounding
    return o, lse, tol, ds


def close(got, want, tol, what):
    assert not torch.isnan(got).any(), f"NaN in {what}"
    err = (got - want).abs()
    err = torch.where(got == want, torch.zeros_like(err), err)               # equal infinities
    bad = err > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(err[bad].max()):.3g} "
                           f"where {float(tol.expand_as(err)[bad].max()):.3g} is allowed, first at {bad.nonzero()[0].tolist()}")
