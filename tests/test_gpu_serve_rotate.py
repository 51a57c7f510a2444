"""GPU parity of norms and rotary positions of queries and keys (qk_rotate of include/wbserve.h) with
their float64 definition (oracle/serving.py).

Tolerance, from the arithmetic (u = 2^-24, half a float32 step). The sum of D squares is at most 16 + 6
additions deep in a lane and across lanes, with one rounding a square: the norm is within 24 u / 2, its root,
quotient and two products 5 u more, relative. A turn is rounded to float32 once (2^-26 of a turn, 6.3 * 2^-26 <
4 u of a radian) and its sine and cosine by 2 u, the magnitude by u; position * frequency in 64 bits by 2^-51 of
the angle; the two products and their sum by 2 u:
  |y - y*| <= eps/2 |y*| + S ((17 + 4 + 2 + 1 + 2) u + 2^-51 |angle|) (1 + eps/2),
S the size of the two terms (of the one, in columns that are not turned), and, for float16, half its
smallest step, 2^-25.
"""
import math

import numpy as np
import pytest

from oracle import serving as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def check(got, x, weight, eps, positions, freqs, interleaved, magnitude):
    kind = got.dtype
    got, x = got.double().cpu().numpy(), x.double().cpu().numpy()
    w = None if weight is None else weight.double().cpu().numpy()
    want, size = O.rotate(x, w, eps, positions, freqs, interleaved, magnitude)
    half = torch.finfo(kind).eps / 2
    angle = np.max(np.abs(np.asarray(positions, np.float64))[:, None, None] * np.max(np.abs(freqs), initial=0), initial=0)
    tol = half * np.abs(want) + size * (26 * U + 2.0 ** -51 * angle) * (1 + half)
    tol += 2.0 ** -25 if kind == torch.float16 else 2.0 ** -140
    err = np.abs(got - want)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4])
    return float((err / tol).max(initial=0))


def run(dtype, N, Hq, H, D, rot, norm=True, interleaved=False, magnitude=1.0, slack=0, far=100000, in_place=False, seed=0,
        wide=False, eps=1e-6, scale=1.0, transposed=False):
    import linear_attn_decode_amd as wb
    print(f"[case] rotate {dtype} N={N} Hq={Hq} H={H} D={D} rot={rot} norm={norm} interleaved={interleaved} slack={slack}", flush=True)
    g = torch.Generator().manual_seed(seed)
    kind = TYPES[dtype]
    rows = (scale * torch.randn((N, (Hq + H) * D + slack), generator=g)).to(kind).cuda()
    keep = rows.clone()
    q, k = rows[:, :Hq * D].unflatten(1, (Hq, D)), rows[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
    q0, k0 = keep[:, :Hq * D].unflatten(1, (Hq, D)), keep[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
    freqs = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    positions = torch.randint(-5, far, (N,), generator=g)
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(kind).cuda() if norm else None for _ in range(2))
    if in_place:
        qo, ko = q, k
        out = {}
    else:
        qo, ko = (torch.full((N, h, D), 7.0, dtype=kind, device="cuda") for h in (Hq, H))
        if transposed:
            qo, ko = (torch.full((h, N, D), 7.0, dtype=kind, device="cuda").transpose(0, 1) for h in (Hq, H))
        out = dict(q_out=qo, k_out=ko)
    wb.qk_rotate(q, k, positions.cuda() if wide else positions.int().cuda(), freqs.cuda(), q_weight=qw, k_weight=kw, eps=eps,
                 interleaved=interleaved, magnitude=magnitude, **out)
    torch.cuda.synchronize()
    args = (eps, positions.numpy(), freqs.numpy(), interleaved, magnitude)
    worst = max(check(qo, q0, qw, *args), check(ko, k0, kw, *args))
    print(f"[worst] {worst:.3f} of the bound", flush=True)
    if in_place:
        assert torch.equal(rows[:, (Hq + H) * D:], keep[:, (Hq + H) * D:])          # the other columns
    else:
        assert torch.equal(rows.view(torch.uint8), keep.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (256, 64), (80, 40), (96, 24), (192, 48), (128, 2), (128, 0), (8, 8),
                                   (1024, 1024), (576, 64)])
def test_heads(dtype, interleaved, D, rot):
    run(dtype, 7, 3, 2, D, rot, norm=True, interleaved=interleaved, seed=D)
    run(dtype, 7, 3, 2, D, rot, norm=False, interleaved=interleaved, magnitude=1.3, seed=D + 1, wide=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot", [(1, 0), (3, 2), (7, 4), (81, 80), (100, 100), (513, 512), (1023, 6), (1000, 1000)])
def test_odd_heads_and_unaligned_rows(dtype, D, rot):
    run(dtype, 5, 2, 1, D, rot, interleaved=False, seed=D, slack=1)
    run(dtype, 5, 2, 1, D, rot, interleaved=True, seed=D, slack=3, in_place=True)


@pytest.mark.parametrize("N,Hq,H", [(1, 1, 1), (1, 32, 8), (2, 40, 40), (300, 32, 8), (5000, 16, 2), (20000, 3, 1)])
def test_tokens_and_heads(N, Hq, H):
    run("bf16", N, Hq, H, 128, 128, seed=N)
    run("bf16", N, Hq, H, 64, 32, interleaved=True, in_place=True, slack=64, seed=N + 1)


def test_transposed_outputs():
    run("f16", 9, 4, 2, 64, 64, transposed=True)


def test_keys_may_be_absent():
    import linear_attn_decode_amd as wb
    g = torch.Generator().manual_seed(1)
    q = torch.randn((5, 3, 64), generator=g)
    freqs, at = wb.rotary_frequencies(64), torch.tensor([0, 1, 2, 3, 10 ** 9]).cuda()
    out = torch.empty((5, 3, 64), device="cuda")
    wb.qk_rotate(q.cuda(), None, at, freqs, q_out=out)
    torch.cuda.synchronize()
    check(out, q, None, 0, at.cpu().numpy(), freqs.cpu().numpy(), False, 1.0)
    assert torch.equal(out[0].cpu(), q[0])                         # position 0 turns nothing


def test_no_tokens():
    import linear_attn_decode_amd as wb
    z = torch.zeros((0, 2, 64), device="cuda")
    wb.qk_rotate(z, z, torch.zeros(0, dtype=torch.int32, device="cuda"), wb.rotary_frequencies(64))
    torch.cuda.synchronize()


@pytest.mark.parametrize("scale,eps", [(2.0 ** 100, 1e-6), (2.0 ** 120, 0.0), (2.0 ** -70, 0.0), (2.0 ** -120, 0.0),
                                       (2.0 ** -70, 1e-37), (2.0 ** -70, 1e-6)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 81, 1024])
def test_norms_of_rows_whose_squares_leave_the_range(dtype, D, scale, eps):
    run(dtype, 4, 2, 1, D, 32, scale=scale, eps=eps, seed=3)


def test_rows_of_zeros_infinities_and_nan():
    import linear_attn_decode_amd as wb
    x = torch.ones((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[0] = 0
    x[1, 0, 3] = math.inf
    x[2, 0, 5] = math.nan
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    wb.qk_rotate(x, None, torch.arange(4, device="cuda"), wb.rotary_frequencies(32), q_weight=w, eps=0.0, q_out=out)
    torch.cuda.synchronize()
    assert (out[0] == 0).all()
    assert torch.isnan(out[1, 0, [3, 19]]).all() and (out[1, 0, 32:] == 0).all() and (out[1, 0, 4:16] == 0).all()
    assert torch.isnan(out[2]).all()
    assert torch.isfinite(out[3]).all()


@pytest.mark.parametrize("far", [2 ** 31 - 1, 10 ** 6])
def test_far_positions(far):
    import linear_attn_decode_amd as wb
    x = torch.ones((3, 1, 128), device="cuda")
    at = torch.tensor([far, -far, far - 1])
    freqs = wb.rotary_frequencies(128, base=500000.0, factor=8.0, context=8192)
    out = torch.empty_like(x)
    wb.qk_rotate(x, None, at.int().cuda(), freqs, q_out=out)
    torch.cuda.synchronize()
    check(out, x, None, 0, at.numpy(), freqs.cpu().numpy(), False, 1.0)


def test_more_tokens_than_a_launch_holds():
    """2^25 + 3 tokens of one head of 2 columns: a wavefront each, past 2^31 work-items."""
    import linear_attn_decode_amd as wb
    n = 2 ** 25 + 3
    x = torch.ones((n, 1, 2), dtype=torch.bfloat16, device="cuda")
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    freqs = torch.tensor([math.pi / 2], dtype=torch.float64, device="cuda")       # quarter turns
    wb.qk_rotate(x, None, at, freqs)
    want = torch.tensor([[1, 1], [-1, 1], [-1, -1], [1, -1]], dtype=torch.bfloat16, device="cuda")
    assert torch.equal(x[:, 0], want[at.long() % 4])


def test_frequencies():
    import linear_attn_decode_amd as wb
    f = wb.rotary_frequencies(64, device="cpu").numpy()
    assert np.allclose(f, [10000.0 ** (-i / 32) for i in range(32)], rtol=1e-15)
    assert np.allclose(wb.rotary_frequencies(64, factor=4.0, device="cpu").numpy(), f / 4, rtol=1e-15)
    s = wb.rotary_frequencies(64, factor=4.0, context=2048, slow=1.0, fast=16.0, device="cpu").numpy()
    turns = 2048 * f / (2 * math.pi)
    assert (s[turns >= 16] == f[turns >= 16]).all() and np.allclose(s[turns <= 1], f[turns <= 1] / 4, rtol=1e-15)
    mid = (turns > 1) & (turns < 16)
    keep = (turns[mid] - 1) / 15
    assert mid.any() and np.allclose(s[mid], f[mid] * (keep + (1 - keep) / 4), rtol=1e-14)
