"""Rotary positions and their gradient (fmha_rope) on the GPU against the
formula in 64 bits."""
import math

import pytest
import torch

from tests import cache_util as cu
from tests import page_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_attention_forward_02_gb300 import build, fmha
    build.build()
    fmha.lib()
    return fmha


def check(got, x, inv_freq, pos, interleaved, magnitude, transpose, dtype):
    y, tol = pu.rope(x.cpu(), inv_freq.cpu(), pos, interleaved, magnitude, transpose)
    if dtype == "e4m3":
        y = y.clamp(-448, 448)
    tol = tol + (y.abs() + tol) * cu.HALF[dtype] + cu.SUBHALF[dtype]
    r = 2 * len(inv_freq)
    if dtype != "e4m3":                                   # behind rot nothing is rounded
        tol[..., r:] = 0
    cu.close(cu.f64(got.cpu()), y, tol, "turned elements")


CASES = {                                                 # B, S, H, H_k, D, rot, far, out
    "one_token": (1, 1, 1, 1, 128, 128, 0, None),
    "one_pair": (1, 3, 2, 1, 8, 2, 7, None),
    "decode_far": (33, 1, 32, 8, 128, 128, (1 << 31) - 40, None),
    "odd_length": (2, 333, 5, 3, 64, 64, 1 << 20, None),
    "part": (2, 65, 8, 2, 128, 32, 5000, None),
    "part_unaligned": (2, 37, 3, 1, 96, 24, 5000, None),
    "scalar": (1, 50, 3, 2, 34, 18, 100, None),
    "largest_head": (1, 9, 2, 2, 256, 256, 100, None),
    "many_tokens": (3, 1100, 6, 2, 64, 48, 0, None),
    "no_keys": (2, 20, 4, 0, 128, 64, 10, None),
    "to_e4m3": (2, 77, 4, 2, 128, 128, 3000, torch.float8_e4m3fn),
    "to_e4m3_scalar": (1, 21, 2, 1, 20, 10, 30, torch.float8_e4m3fn),
}


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", CASES)
def test_rope(fm, name, dtype, interleaved, transpose):
    B, S, H, H_k, D, rot, far, out = CASES[name]
    g = torch.Generator().manual_seed(len(name))
    q = cu.draw(g, (B, S, H, D), dtype, 200.0 if out else 2.0).cuda()
    k = cu.draw(g, (B, S, H_k, D), dtype).cuda() if H_k else None
    pos = torch.randint(0, far + 1, (B, S), generator=g).to(torch.int32) if far else None
    if transpose and out:
        pytest.skip("gradients keep their type")
    inv_freq, magnitude = fm.rope_frequencies(rot, base=10000.0, scaling="by_parts", factor=4.0, trained=2048, device="cuda")
    f = fm.rope_bwd if transpose else fm.rope
    kw = {} if transpose else dict(out_dtype=out)
    yq, yk = f(q, k, inv_freq, positions=pos.cuda() if far else None, interleaved=interleaved, magnitude=magnitude, **kw)
    at = pos if far else torch.arange(S).expand(B, S)
    odt = "e4m3" if out else dtype
    check(yq, q, inv_freq, at, interleaved, magnitude, transpose, odt)
    if H_k:
        check(yk, k, inv_freq, at, interleaved, magnitude, transpose, odt)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("token_pad", [0, 24])
def test_pieces_of_a_projection_in_place(fm, interleaved, token_pad):
    B, S, H, H_k, D = 2, 45, 6, 2, 64
    g = torch.Generator().manual_seed(3)
    rows = cu.draw(g, (B, S, (H + 2 * H_k) * D + token_pad), "bf16").cuda()
    was = rows.clone()
    part = lambda t, a, h: t[..., a * D:(a + h) * D].unflatten(-1, (h, D))
    q, k = part(rows, 0, H), part(rows, H, H_k)
    inv_freq, _ = fm.rope_frequencies(48, device="cuda")
    yq, yk = fm.rope(q, k, inv_freq, interleaved=interleaved, q_out=q, k_out=k)
    at = torch.arange(S).expand(B, S)
    check(yq, part(was, 0, H), inv_freq, at, interleaved, 1.0, False, "bf16")
    check(yk, part(was, H, H_k), inv_freq, at, interleaved, 1.0, False, "bf16")
    assert torch.equal(rows[..., (H + H_k) * D:], was[..., (H + H_k) * D:])


def test_head_major_and_odd_strides(fm):
    B, S, H, D = 2, 31, 3, 64
    g = torch.Generator().manual_seed(4)
    q = cu.draw(g, (B, H, S, D), "f16").cuda().transpose(1, 2)
    k = cu.draw(g, (B, S, H, D + 3), "f16").cuda()[..., 1:D + 1]          # rows at odd addresses
    inv_freq, _ = fm.rope_frequencies(D, device="cuda")
    out = cu.sentinel((B, H, S, D), torch.float16).transpose(1, 2)
    yq, yk = fm.rope(q, k, inv_freq, q_out=out)
    at = torch.arange(S).expand(B, S)
    check(yq, q, inv_freq, at, False, 1.0, False, "f16")
    check(yk, k, inv_freq, at, False, 1.0, False, "f16")
    assert yq.data_ptr() == out.data_ptr()


def test_broadcast_input(fm):
    g = torch.Generator().manual_seed(5)
    one = cu.draw(g, (1, 1, 4, 64), "bf16").cuda()
    inv_freq, _ = fm.rope_frequencies(64, device="cuda")
    y, _ = fm.rope(one.expand(2, 9, 4, 64), None, inv_freq)
    check(y, one.expand(2, 9, 4, 64), inv_freq, torch.arange(9).expand(2, 9), False, 1.0, False, "bf16")


@pytest.mark.parametrize("D,rot", [(64, 32), (34, 18)])
def test_rows_without_a_position_are_left_out(fm, D, rot):
    g = torch.Generator().manual_seed(6)
    q = cu.draw(g, (11, 3, D), "bf16").cuda()
    pos = torch.tensor([4, -1, 0, 7, -5, 9, 1, 2, 3, -1, -1], dtype=torch.int32)
    inv_freq, _ = fm.rope_frequencies(rot, device="cuda")
    out = cu.sentinel(q.shape, torch.bfloat16)
    fm.rope(q, None, inv_freq, positions=pos.cuda(), q_out=out)
    some = pos >= 0
    check(out[some.cuda()], q[some.cuda()], inv_freq, pos[some], False, 1.0, False, "bf16")
    assert cu.untouched(out[~some.cuda()])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(fm, interleaved):
    """The map is linear: <dy, f(x + h e) - f(x - h e)> / 2h = <dx, e>, in the
    64-bit form; fmha_rope's transpose is held to that form above, and here to
    <dy, f(e)> for f as the GPU computes it."""
    g = torch.Generator().manual_seed(7)
    S, H, D, rot = 13, 2, 32, 20
    e, dy = (torch.randn((1, S, H, D), generator=g).to(torch.float16) for _ in range(2))
    inv_freq, m = fm.rope_frequencies(rot, device="cuda")
    m = 1.25
    at = torch.arange(S).expand(1, S)
    h = 2.0 ** -10
    x = torch.randn((1, S, H, D), generator=g).double()
    f = lambda v: pu.rope(v, inv_freq.cpu(), at, interleaved, m)[0]
    slope = ((f(x + h * e.double()) - f(x - h * e.double())) / (2 * h) * dy.double()).sum()
    dx, _ = fm.rope_bwd(dy.cuda(), None, inv_freq, interleaved=interleaved, magnitude=m)
    ye, _ = fm.rope(e.cuda(), None, inv_freq, interleaved=interleaved, magnitude=m)
    a = (dx.double().cpu() * e.double()).sum()
    b = (ye.double().cpu() * dy.double()).sum()
    # every element of dx and f(e) rounded by 2^-11 at most
    tol = 2.0 ** -10 * float((dx.double().cpu().abs() * e.double().abs()).sum() + (ye.double().cpu().abs() * dy.double().abs()).sum())
    assert abs(a - slope) <= tol and abs(b - slope) <= tol


def test_attention_on_turned_tensors_depends_on_distances_alone(fm):
    """rope, forward and backward, as a training step runs them: with all
    positions shifted, O and the gradients of the unturned q and k stay."""
    g = torch.Generator().manual_seed(8)
    B, S, H, D = 2, 200, 2, 64
    q, k, v, do = (cu.draw(g, (B, S, H, D), "bf16").cuda() for _ in range(4))
    inv_freq, _ = fm.rope_frequencies(D, device="cuda")
    got = []
    for shift in (0, 100000):
        pos = (torch.arange(S) + shift).to(torch.int32).expand(B, S).contiguous().cuda()
        qr, kr = fm.rope(q, k, inv_freq, positions=pos)
        o, lse = fm.fwd(qr, kr, v, mask="causal")
        dq, dk, dv = fm.bwd(qr, kr, v, o, do, lse, mask="causal")
        dq, dk = fm.rope_bwd(dq, dk, inv_freq, positions=pos)
        got.append([t.double() for t in (o, dq, dk, dv)])
    # turned tensors are rounded to bf16 in another direction: 2^-8 of an
    # element, of either factor, in scores of up to |q||k| / 8
    for a, b in zip(*got):
        rel = ((a - b).norm() / a.norm()).item()
        assert rel < 8 * 2.0 ** -8, rel
    # and the formula's gradient, by torch's own differentiation in 64 bits
    qd, kd, vd = (t.double().cpu().requires_grad_() for t in (q, k, v))
    ang = torch.arange(S).double()[:, None, None] * inv_freq.cpu()
    c, s = torch.cos(ang), torch.sin(ang)
    turn = lambda x: torch.cat([x[..., :D // 2] * c - x[..., D // 2:] * s, x[..., D // 2:] * c + x[..., :D // 2] * s], -1)
    x = torch.einsum("bihd,bjhd->bhij", turn(qd), turn(kd)) / math.sqrt(D)
    x = x.masked_fill(~torch.ones((S, S), dtype=torch.bool).tril(), -math.inf)
    torch.einsum("bhij,bjhd->bihd", torch.softmax(x, -1), vd).backward(do.double().cpu())
    for a, b in zip(got[0][1:], (qd.grad, kd.grad, vd.grad)):
        rel = ((a.cpu() - b).norm() / b.norm()).item()
        assert rel < 8 * 2.0 ** -8, rel
