"""The paged-cache operators as a server runs them together: plan, rope, write,
attention; prompts, single tokens, drafts that are taken back, requests that
end and new ones in their pages."""
import math
import random

import pytest
import torch

from tests import cache_util as cu
from tests import page_util as pu

pytestmark = pytest.mark.gpu
H, H_k, D, P = 8, 2, 128, 16


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_attention_forward_02_gb300 import build, fmha
    build.build()
    fmha.lib()
    return fmha


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Server:
    """B requests over a small cache; keeps what every cached token's key and value were."""

    def __init__(self, fm, B, n_pages, width, dtype="bf16", seed=0):
        self.fm, self.B, self.dt, self.dtype = fm, B, cu.DTYPES[dtype], dtype
        self.gen, self.rng = torch.Generator().manual_seed(seed), random.Random(seed)
        self.entry = self.rng.sample(range(B), B)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.free, self.n_free, self.n_pages = i32(self.rng.sample(range(n_pages), n_pages)), i32([n_pages]), n_pages
        self.seqlen, self.idx = i32([0] * B), i32(self.entry)
        nan = lambda: torch.full((n_pages, H_k, P, D), 0x7F, dtype=torch.uint8, device="cuda").view(pu.E4M3)
        self.pool = [nan(), nan(), torch.zeros((n_pages, H_k), device="cuda"), torch.zeros((n_pages, H_k), device="cuda")]
        self.inv_freq, self.magnitude = fm.rope_frequencies(64, scaling="by_parts", factor=4.0, trained=64, device="cuda")
        self.k, self.v = [[] for _ in range(B)], [[] for _ in range(B)]       # turned keys and values, by token

    def step(self, n_new, pad=2):
        fm, N = self.fm, sum(max(0, n) for n in n_new) + pad
        was = self.seqlen.tolist()
        slots, pos, cu_new, new_len = fm.page_plan(self.seqlen, i32(n_new), self.table, self.free, self.n_free, page_size=P,
                                                   max_tokens=N, batch_idx=self.idx, new_seqlen=self.seqlen)
        got = new_len.tolist()
        for b, n in enumerate(n_new):
            if n < 0:
                del self.k[b][got[b]:], self.v[b][got[b]:]
        # one projection's rows: q, k and v are pieces of them
        rows = torch.randn((N, (H + 2 * H_k) * D), generator=self.gen).to(self.dt).cuda()
        rows[:, :H * D] *= 2
        piece = lambda a, h: rows[:, a * D:(a + h) * D].unflatten(1, (h, D))
        q, k, v = piece(0, H), piece(H, H_k), piece(H + H_k, H_k)
        plain = k.clone()
        fm.rope(q, k, self.inv_freq, positions=pos, magnitude=self.magnitude, q_out=q, k_out=k)
        fm.page_write(k, v, slots, *self.pool)
        out, lse = cu.sentinel((N, H, D), self.dt), cu.sentinel((N, H), torch.float32)
        fm.page_fwd(q.contiguous(), *self.pool, self.table, self.seqlen, cu_q=cu_new, max_q=max(1, *n_new), batch_idx=self.idx, out=out,
                    lse=lse)
        torch.cuda.synchronize()
        assert fm.device_status(reset=True) == 0
        at = 0
        for b, n in enumerate(n_new):
            if n > 0 and got[b] == was[b] + n:
                want, tol = pu.rope(plain[at:at + n].cpu(), self.inv_freq.cpu(), torch.arange(was[b], was[b] + n), False, self.magnitude)
                turned = k[at:at + n].cpu()
                cu.close(cu.f64(turned), want, tol + (want.abs() + tol) * cu.HALF[self.dtype], f"turned keys of {b}")
                self.k[b] += list(turned)
                self.v[b] += list(v[at:at + n].cpu())
            assert got[b] == len(self.k[b])
            at += max(0, n)
        self.check(q.cpu(), out.cpu(), lse.cpu(), n_new, got, was, cu_new.tolist())

    def check(self, q, out, lse, n_new, lens, was, cu_new):
        codes = [self.pool[x].cpu().view(torch.uint8) for x in (0, 1)]
        scales = [self.pool[x].cpu().double() for x in (2, 3)]
        used = []
        for b, L in enumerate(lens):
            ids = self.table[self.entry[b], :pu.up(L, P)].cpu().long()
            used += ids.tolist()
            cached = []
            for x, tokens in ((0, self.k[b]), (1, self.v[b])):
                c = pu.VALUES[codes[x][ids].transpose(0, 1).reshape(H_k, -1, D).long()][:, :L]
                s = scales[x][ids].T.repeat_interleave(P, 1)[:, :L]
                if L:
                    # a value is rounded to e4m3, and again where its page's scale grew
                    want = torch.stack(tokens).double().transpose(0, 1)
                    cu.close(c * s[..., None], want, want.abs() * 2 * 2.0 ** -4 * 1.07 + s[..., None] * 2.0 ** -9, f"cache of {b}")
                cached.append((c, s))
            n = max(0, n_new[b])
            if n == 0 or L != was[b] + n:
                continue
            see = torch.arange(L)[None] <= was[b] + torch.arange(n)[:, None]
            for g in range(H_k):
                h = slice(g * H // H_k, (g + 1) * H // H_k)
                (kc, ks), (vc, vs) = cached
                o, l, tol, tl = pu.attend(cu.f64(q[cu_new[b]:cu_new[b] + n][:, h]), kc[g], ks[g], vc[g], vs[g], see, D ** -0.5, 1.0,
                                          self.dtype, True)
                cu.close(cu.f64(out[cu_new[b]:cu_new[b] + n][:, h]), o, tol, f"O of {b}")
                cu.close(lse[cu_new[b]:cu_new[b] + n][:, h].double(), l, tl, f"LSE of {b}")
        assert len(set(used)) == len(used), "a page has two owners"
        n = int(self.n_free)
        assert sorted(used + self.free[:n].tolist()) == list(range(self.n_pages)), "a page is lost or doubled"
        assert cu.untouched(out[cu_new[-1]:]) and cu.untouched(lse[cu_new[-1]:])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_server(fm, dtype):
    s = Server(fm, 4, 40, 12, dtype)
    for n_new in ([50, 17, 0, 3], [1, 1, 1, 1], [4, 4, 0, 4], [-3, -2, 0, 0], [1, 0, 90, 1], [-48, 1, 1, 1], [33, 1, 1, 1], [5, -20, 0, 1],
                  [1, 60, 1, 1], [1, 1, 1, 1]):
        s.step(n_new)


def test_requests_that_do_not_fit_wait(fm):
    s = Server(fm, 3, 6, 8, seed=1)
    s.step([60, 20, 40])                                  # 4 + 2 pages; the third gets none
    assert s.seqlen.tolist() == [60, 20, 0]
    s.step([1, 1, 40])
    s.step([-61, 1, 40])                                  # the first has ended
    assert s.seqlen.tolist() == [0, 22, 40]


def test_decode_in_a_graph(fm):
    """Plan, rope, write and attention captured once, everything in place, and
    replayed against the same calls run eagerly."""
    B, steps = 5, 40
    got = []
    for graph in (False, True):
        s = Server(fm, B, 60, 10, seed=2)
        s.step([30, 1, 16, 47, 5])
        g = torch.Generator().manual_seed(3)
        feed = torch.randn((steps, B, (H + 2 * H_k) * D), generator=g).to(s.dt).cuda()
        rows, ones = torch.empty_like(feed[0]), i32([1] * B)
        slots, pos, cu_new = torch.empty_like(ones), torch.empty_like(ones), torch.empty(B + 1, dtype=torch.int32, device="cuda")
        out, lse = torch.empty((B, H, D), dtype=s.dt, device="cuda"), torch.empty((B, H), device="cuda")
        ws = torch.empty(fm.fmha_page_workspace_size(1, H, H_k), dtype=torch.uint8, device="cuda")
        piece = lambda a, h: rows[:, a * D:(a + h) * D].unflatten(1, (h, D))
        q, k, v = torch.empty((B, H, D), dtype=s.dt, device="cuda"), piece(H, H_k), piece(H + H_k, H_k)

        def step():
            fm.page_plan(s.seqlen, ones, s.table, s.free, s.n_free, page_size=P, batch_idx=s.idx, slots=slots, positions=pos,
                         cu_new=cu_new, new_seqlen=s.seqlen)
            fm.rope(piece(0, H), k, s.inv_freq, positions=pos, magnitude=s.magnitude, q_out=q, k_out=k)
            fm.page_write(k, v, slots, *s.pool)
            fm.page_fwd(q, *s.pool, s.table, s.seqlen, batch_idx=s.idx, out=out, lse=lse, workspace=ws)

        if graph:
            keep = [t.clone() for t in (s.table, s.free, s.n_free, s.seqlen, *s.pool)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            rows.copy_(feed[0])
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
            for t, was in zip((s.table, s.free, s.n_free, s.seqlen, *s.pool), keep):
                t.view(torch.uint8).copy_(was.view(torch.uint8)) if t.dtype == pu.E4M3 else t.copy_(was)
        outs = []
        for i in range(steps):
            rows.copy_(feed[i])
            captured.replay() if graph else step()
            outs += [out.clone(), lse.clone()]
        torch.cuda.synchronize()
        assert fm.device_status(reset=True) == 0
        got.append(outs + [s.table, s.free[:int(s.n_free)], s.seqlen, s.pool[2], s.pool[3]])
        ids = [s.table[s.entry[b], :pu.up(int(s.seqlen[b]), P)].long() for b in range(B)]
        got[-1] += [s.pool[x].view(torch.uint8)[torch.cat(ids)] for x in (0, 1)]
    for a, b in zip(*got):
        assert torch.equal(a, b)
