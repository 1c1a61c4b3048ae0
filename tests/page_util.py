"""Plain forms of the paged-cache operators on the CPU, in whole numbers and 64
bits, for the tests."""
from __future__ import annotations

import torch

from tests import cache_util as cu

E4M3 = torch.float8_e4m3fn
VALUES = torch.arange(256, dtype=torch.uint8).view(E4M3).float().double()      # of every code


def up(a, b):
    return -(-a // b)


def plan(seqlen, n_new, table, free_list, n_free, page, rows, entry=None):
    """The plan's outputs from lists; table (list of lists) and free_list are changed."""
    B, width = len(seqlen), len(table[0])
    entry = entry or list(range(B))
    stack = list(free_list[:n_free])
    new_len, slots, pos, cu_new = list(seqlen), [-1] * rows, [-1] * rows, [0]
    for b, n in enumerate(n_new):
        if n < 0:
            keep = max(0, seqlen[b] + n)
            stack += [table[entry[b]][i] for i in range(up(keep, page), up(seqlen[b], page))]
            new_len[b] = keep
    for i, x in enumerate(stack):                       # where the stack reached, its pages stay written
        free_list[i] = x
    stopped = False
    for b, n in enumerate(n_new):
        L = seqlen[b]
        fits = True
        if n >= 0:
            fits = L + n <= width * page
            need = up(L + n, page) - up(L, page) if fits else 0
            if need > len(stack) or (need and stopped):
                stopped = fits = False
                stopped = True
            elif fits:
                for i in range(need):
                    table[entry[b]][up(L, page) + i] = stack.pop()
                new_len[b] = L + n
        for t in range(max(n, 0)):
            i = cu_new[-1] + t
            if i < rows:
                pos[i] = L + t
                slots[i] = table[entry[b]][(L + t) // page] * page + (L + t) % page if fits else -1
        cu_new.append(min(rows, cu_new[-1] + max(n, 0)))
    return slots, pos, cu_new, new_len, len(stack)


def rope(x, inv_freq, pos, interleaved, magnitude, transpose=False):
    """Turned x [..., heads, D] in 64 bits, and the bound on what fp32 may be off by."""
    r = 2 * len(inv_freq)
    ang = pos.double()[..., None, None] * inv_freq.double()
    c, s = torch.cos(ang) * magnitude, torch.sin(ang) * magnitude * (-1 if transpose else 1)
    x = x.double()
    i = torch.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    y, tol = x.clone(), torch.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    # sine and cosine: the angle is off by 2^-25 half turns, 9.4e-8, and they by
    # 2^-23 more; three fp32 roundings behind them
    both = (x[..., a].abs() + x[..., b].abs()) * abs(magnitude) * 2.0 ** -21
    tol[..., a] = tol[..., b] = both
    return y, tol


def exponent(a):
    """Least e in [-60, 60] with a <= 448 * 2^e."""
    e = -60
    while e < 60 and a > 448.0 * 2.0 ** e:
        e += 1
    return e


def codes(x):
    """e4m3 codes of 64-bit values that 32 bits hold: nearest even, saturating."""
    return x.clamp(-448, 448).float().to(E4M3).view(torch.uint8)


def write(new, slots, pages, scale):
    """new [N, H_k, 128] into pages (uint8 codes [n, H_k, P, 128]) and scale, both changed."""
    P, x = pages.shape[2], new.double()
    i = 0
    while i < len(slots):
        if slots[i] < 0 or slots[i] >= pages.shape[0] * P:
            i += 1
            continue
        n, p, off = 1, slots[i] // P, slots[i] % P
        while i + n < len(slots) and off + n < P and (slots[i + n] < 0 or slots[i + n] == slots[i] + n):
            n += 1
        for g in range(pages.shape[1]):
            live = torch.tensor(slots[i:i + n]) >= 0
            run = x[i:i + n, g][live]
            top = run.abs().nan_to_num(nan=0.0, posinf=float("inf")).max().item()
            s, old = 2.0 ** exponent(top), scale[p, g].item()
            if off > 0:
                if s > old:
                    pages[p, g, :off] = codes(VALUES[pages[p, g, :off].long()] * (old / s))
                s = max(s, old)
            pages[p, g, off:off + n][live] = codes(run / s)
            scale[p, g] = s
        i += n


def draw_pages(gen, n_pages, H_k, P, lo=-8, hi=-4):
    """Codes and power-of-two scales of a cache whose values are about one."""
    c = cu.draw(gen, (n_pages, H_k, P, 128), "e4m3", 64.0)
    s = torch.exp2(torch.randint(lo, hi, (n_pages, H_k), generator=gen).float())
    return c, s


def attend(q, kc, ks, vc, vs, see, scale, out_scale, dtype, chunk=False):
    """One sequence and kv head in 64 bits: q [n, G, 128]; kc, vc codes' values
    [L, 128]; ks, vs their scales [L]; see [n, L]; chunk: sequences of many rows, which a kernel of their own takes.  Returns O, LSE and the bounds on
    their errors."""
    n, G, _ = q.shape
    L = kc.shape[0]
    keys, vals = kc * ks[:, None], vc * vs[:, None]
    if L == 0 or n == 0:
        return torch.zeros(n, G, 128).double(), torch.full((n, G), -float("inf")).double(), torch.zeros(n, G, 128).double(), \
            torch.zeros(n, G).double()
    x = torch.einsum("tgd,kd->tgk", q, keys) * scale
    x = x.masked_fill(~see[:, None, :], -float("inf"))
    lse = torch.logsumexp(x, -1)
    empty = lse == -float("inf")
    w = torch.exp(x - torch.where(empty, 0.0, lse)[..., None])
    o = torch.einsum("tgk,kd->tgd", w, vals) * out_scale
    seen = see[:, None, :].double()
    # a score: 128 products summed in fp32, each addition off by 2^-23 of the
    # partial sum; elements of q by 2^-21 (chunk: 2^-17) of the row's largest; then a few fp32
    # roundings of the score, of its exponential and of the sums
    a = (torch.einsum("tgd,kd->tgk", q.abs(), keys.abs()) * scale * seen).amax(-1)
    top = q.abs().amax(-1)
    ds = (a * 134 * 2.0 ** -23 + top * 2.0 ** (-17 if chunk else -21) * (keys.abs().sum(-1)[None, None] * seen).amax(-1) * scale +
          lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -21 + 1e-5)
    # a weight: two terms of four bits (2^-8; f16 three, 2^-12) from f16's eleven (2^-11;
    # chunk: these, and 2^-12 for the sums of up to 2^10 products, each off by 2^-23 of
    # the partial one); and where the terms end, 2^-14 where the largest weight is 2^4 or more
    ab = torch.einsum("tgk,kd->tgd", w, vals.abs()) * abs(out_scale)
    low = (w * vs).amax(-1, keepdim=True) * torch.einsum("tgk,kd->tgd", seen.expand(n, G, L), vc.abs()) * abs(out_scale)
    tol = ab * (2.0 ** (-12 if chunk or dtype == "f16" else -8) + 2.0 ** -11 + 2 * ds[..., None]) + low * 2.0 ** -18
    tol = tol + (o.abs() + tol) * cu.HALF[dtype] + cu.SUBHALF[dtype]
    return o, lse, tol, ds
