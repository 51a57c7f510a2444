"""kv_attend_chunk (include/wbserve.h) over scores far from 0, whole and split requests.

Keys and queries are chosen so that a score, base + step, is a float32 number and so is every partial sum
of its products: the scores are exact, and what remains is the softmax's own error (u = 2^-24). With d the
score's distance from the largest, an exponent is d * (scale log2 e), within 4 u |d|, or, where the
reference's own product is small, base * (scale log2 e) under 2^8, within 2^-15 (the product's rounding and
the sum's, 2^-17 each, for the weight and for the reference that it is joined to); the exponential adds 2^-22:
e = 2^-15 + 2^-22 + 4 u |d|. The weight's rounding r is 2^-8 in bfloat16, 2^-11 in float16 (and 2^-36 of the
largest), sums take 16 tokens a step, the output is rounded once:
  |o - o*| <= eps/2 |o*| + W (2 E + r + 2 (96 + n/16) u) (1 + eps/2),  W = sum p|v|,
  |lse - lse*| <= E + (96 + n/16) u + 4 u |lse*|,  E = the largest e of a weight that counts (d <= 40).
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def attend(kv, qt, D, base, steps, m, scale, values):
    """m new tokens over scores (base + steps[t]) * scale; q is (1, 1, 0, ...), the keys (base, step, 0, ...) with
    the base's power of two in q."""
    import linear_attn_decode_amd as wb
    page, n = 16, len(steps)
    pages = -(-n // page)
    q = torch.zeros((m, 2, D), device="cuda")
    k = torch.zeros((pages * page, 1, D), device="cuda")
    up = 2.0 ** (math.frexp(abs(base))[1] // 2) if base else 1.0         # (a float16 key holds half of the power)
    q[..., 0], q[..., 1] = up, 1
    k[:n, 0, 0], k[:n, 0, 1] = base / up, torch.tensor(steps, dtype=torch.float32)
    v = torch.zeros((pages * page, 1, D), device="cuda")
    v[:n, 0] = values
    paged = lambda x: x.view(pages, page, 1, D).transpose(1, 2).contiguous()
    ones = torch.ones((pages, 1, page), device="cuda") if kv == "e4m3" else None
    kc, vc = paged(k).to(TYPES[kv]), paged(v).to(TYPES[kv])
    assert torch.equal(kc.float(), paged(k)) and torch.equal(q.to(TYPES[qt]).float(), q) and torch.equal(vc.float(), paged(v))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    o = torch.full((m, 2, D), 7.0, dtype=TYPES[qt], device="cuda")
    lse = torch.full((m, 2), 7.0, device="cuda")
    wb.kv_attend_chunk(q.to(TYPES[qt]), kc, vc, i32([list(range(pages))]), i32([n]), i32([0, m]), o, scale=scale, lse=lse,
                       k_scale=ones, v_scale=ones)
    torch.cuda.synchronize()
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def check(kv, qt, D, base, steps, m, scale):
    n = len(steps)
    print(f"[case] far kv={kv} q={qt} D={D} base={base} n={n} m={m} scale={scale}", flush=True)
    g = torch.Generator().manual_seed(n + D)
    values = torch.randint(-8, 9, (n, D), generator=g).float() / 4
    o, lse = attend(kv, qt, D, base, steps, m, scale, values.cuda())
    v = values.double().numpy()
    r = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -8}[kv]
    half = torch.finfo(TYPES[qt]).eps / 2
    s = scale * (base + np.asarray(steps, np.float64))
    for i in range(m):
        seen = n - m + i + 1
        top = s[:seen].max()
        d = top - s[:seen]
        w = np.exp(-d)
        total = w.sum()
        ro, W, rl = w @ v[:seen] / total, w @ np.abs(v[:seen]) / total, top + math.log(total)
        E = 2.0 ** -15 + 2.0 ** -22 + 4 * U * d[d <= 40].max()
        sums = (96 + n / 16) * U
        tol = half * np.abs(ro) + W * (2 * E + r + 2 * sums) * (1 + half) + 2.0 ** -25 + (n * 2.0 ** -36 * 2 if kv == "f16" else 0)
        for h in range(2):
            assert (np.abs(o[i, h] - ro) <= tol).all(), (i, h, o[i, h][:4], ro[:4])
            assert abs(lse[i, h] - rl) <= E + sums + 4 * U * abs(rl), (i, h, lse[i, h], rl)


def rising(n, unit, high):
    """Steps 0, unit, 2 unit by turns, and a few tokens `high` and 2 `high` above them where later tiles begin."""
    steps = [unit * (t % 3) for t in range(n)]
    for at, by in ((n // 3, high), (n // 2 + 5, high), (2 * n // 3, 2 * high)):
        steps[at] = by
    return steps


KINDS = [("bf16", "bf16", 64), ("f16", "f16", 128), ("e4m3", "bf16", 128), ("bf16", "bf16", 256), ("f16", "f16", 256)]


@pytest.mark.parametrize("kv,qt,D", KINDS)
@pytest.mark.parametrize("exponent", [6, 8, 10, 14, 17, 20])
@pytest.mark.parametrize("sign", [1, -1])
def test_common_offsets_of_all_scores(kv, qt, D, exponent, sign):
    """A large number added to every score changes no weight."""
    if kv == "e4m3" and exponent > 14:
        exponent = exponent - 6                      # (up to 448 in a code, and 2^7 in a bfloat16 query)
    unit = 2.0 ** max(-3, exponent - 22)
    check(kv, qt, D, sign * 2.0 ** exponent, rising(200, unit, 4.0), 40, 1.0)


@pytest.mark.parametrize("kv,qt,D", KINDS[:4])
@pytest.mark.parametrize("exponent", [8, 20, 24, 28, 31, 33, 36, 40, 60, 90, 99, 101, 120])
@pytest.mark.parametrize("n,m", [(200, 40), (5000, 3)])
def test_scores_of_any_size(kv, qt, D, exponent, n, m):
    """Scores of 2^exponent, by the scale: only the largest count, however large they are."""
    steps = [float(t % 5) for t in range(n)]
    steps[n // 3] = 6.0                                 # the largest from there on
    for sign in (1, -1):
        check(kv, qt, D, 0.0, steps, m, sign * 2.0 ** (exponent - 2) * 1.25)


@pytest.mark.parametrize("qt", ["bf16", "f16"])
@pytest.mark.parametrize("size", [1e3, 1e9, 1e10, 1e11, 1e15])
def test_agrees_with_kv_attend_on_ordinary_vectors_and_large_scales(qt, size):
    """Random queries and keys: a row's heaviest token is the heaviest of both operators, to its last bit, where the
    scores' distances leave no other a weight."""
    import linear_attn_decode_amd as wb
    print(f"[case] large scale q={qt} {size}", flush=True)
    g = torch.Generator().manual_seed(3)
    R, H, G, D, page, n = 24, 2, 4, 128, 16, 400
    k, v = (torch.randn((R * 25, H, page, D), generator=g).to(TYPES[qt]).cuda() for _ in range(2))
    q = torch.randn((R, H * G, D), generator=g).to(TYPES[qt]).cuda()
    table = torch.arange(R * 25, dtype=torch.int32).view(R, 25).cuda()
    lens = torch.full((R,), n, dtype=torch.int32).cuda()
    one, many = torch.empty_like(q), torch.empty_like(q)
    l1, l2 = (torch.empty((R, H * G), device="cuda") for _ in range(2))
    wb.kv_attend(q, k, v, table, lens, one, scale=size, lse=l1)
    wb.kv_attend_chunk(q, k, v, table, lens, torch.arange(R + 1, dtype=torch.int32).cuda(), many, scale=size, lse=l2)
    torch.cuda.synchronize()
    s = torch.matmul(q.double().view(R, H, G, D), k.view(R, 25, H, page, D).transpose(1, 2).reshape(R, H, n, D).double().transpose(2, 3).contiguous())
    two = s.topk(2, dim=3).values.view(R, H * G, 2) * size
    # (both scores are within (D + 8) u of sum |q k| of these: 200 or so)
    clear = (two[..., 0] - two[..., 1]) > 40 + 2 * (D + 8) * U * 200 * size
    assert clear.float().mean().item() > 0.6
    assert torch.equal(one[clear], many[clear])
    assert (l1 - l2).abs().max().item() <= 2 * (D + 8) * U * 200 * size
