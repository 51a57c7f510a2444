"""GPU parity of attention of chunks of new tokens (kv_attend_chunk of include/wbserve.h) with its
float64 definition (oracle/serving.py).

Tolerance, from the arithmetic (u = 2^-24, half a float32 step). A score is a float32 sum of D exact
products, scaled up to three times (the key's scale, the scale and log2 e): within (D + 8) u
sum|scale q k|; a weight e^{s - ref} adds the rounding of the exponent and of the exponential, 2^-22
together, relative to max(1, |s|). The weights are rounded to the type of the value's operand, by half a
step: r = 2^-8 of each in bfloat16, 2^-11 in float16 (and by half of its smallest step, 2^-25, at 2^11 times
the weight: 2^-36 a token, of a sum of at least 1), or, as two bfloat16 limbs for a float16 query over an
8-bit cache, 2^-16. Sums over tokens take 16 products a step and a
step a tile: (96 + n / 16) u of sum p|v|, and as much for the sum of weights. The output is rounded once:
  |o - o*| <= eps/2 |o*| + W (2 e_s + r + 2 (96 + n/16) u) (1 + eps/2),  W = sum p|v| / sum p,
  |lse - lse*| <= e_s + (96 + n/16) u + 2 u |lse*|,  e_s = (D + 8) u A + 2^-22 max(1, A),
A the largest sum|scale q k|.
"""
import math

import numpy as np
import pytest

from oracle import serving as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def rand(g, *shape, dtype="f32"):
    return torch.randn(shape, generator=g).to(TYPES[dtype])


def stored64(cache, scale):
    x = cache.float().double().cpu().numpy()
    return x if scale is None else x * scale.double().cpu().numpy()[..., None]


def random_cache(g, pages, H, page, D, kv):
    if kv != "e4m3":
        return rand(g, pages, H, page, D, dtype=kv).cuda(), None
    codes = (rand(g, pages, H, page, D) * 100).clamp(-448, 448).to(TYPES[kv])
    return codes.cuda(), ((0.5 + torch.rand((pages, H, page), generator=g)) / 100).cuda()


def make_table(rng, lens, page, pages, width):
    """Every request's pages from a shuffled pool; entries behind a request's last are ids of nobody."""
    order = rng.permutation(pages)
    table = np.full((len(lens), width), 1 << 30, np.int32)
    at = 0
    for r, n in enumerate(lens):
        c = -(-n // page)
        table[r, :c] = order[at:at + c]
        at += c
    return table


def bounds(kv, qt, D, n, ro, rl, W, size, v_max):
    A = max(1.0, size.max(initial=0))
    e_s = (D + 8) * U * A + 2.0 ** -22 * A
    sums = (96 + n / 16) * U
    r = 2.0 ** -16 if kv == "e4m3" and qt == "f16" else 2.0 ** -11 if kv == "f16" else 2.0 ** -8
    half = torch.finfo(TYPES[qt]).eps / 2
    tol = half * np.abs(ro) + W * (2 * e_s + r + 2 * sums) * (1 + half) + 2.0 ** -40
    if qt == "f16":
        tol += 2.0 ** -25                                      # (outputs below the normal numbers)
    if kv == "f16":
        tol += n * 2.0 ** -36 * v_max
    return tol, e_s + sums + 2 * U * np.abs(rl)


def check(o, lse, q, k, v, table, lens, starts, page, scale, window, kv, qt, skip=()):
    o, lse, q = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    worst = 0.0
    for r, n in enumerate(lens):
        rows = slice(starts[r], starts[r + 1])
        if r in skip or starts[r] == starts[r + 1]:
            continue
        t = np.arange(n)
        at = table[r][t // page]
        kr, vr = k[at, :, t % page], v[at, :, t % page]
        ro, rl, W, size = O.attend_chunk(q[rows], kr, vr, scale, window)
        tol, ltol = bounds(kv, qt, q.shape[2], n, ro, rl, W, size, np.abs(vr).max(initial=0))
        err = np.abs(o[rows] - ro)
        assert (err <= tol).all(), (r, n, float(np.nanmax(err / tol)), np.argwhere(~(err <= tol))[:4])
        worst = max(worst, float((err / tol).max()))
        none = np.isneginf(rl)
        assert (np.isneginf(lse[rows]) == none).all(), (r, n)
        assert (np.abs(lse[rows][~none] - rl[~none]) <= ltol[~none]).all(), (r, n)
    return worst


def run(kv, qt, D, H, G, news, pasts, page, window=0, seed=0, strided=False, scale=None, pad=0, spare=2):
    import linear_attn_decode_amd as wb
    print(f"[case] chunk kv={kv} q={qt} D={D} H={H} G={G} new={news[:8]} past={pasts[:8]} R={len(news)} page={page} "
          f"window={window}", flush=True)
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    lens = [a + b for a, b in zip(news, pasts)]
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    pages = sum(-(-n // page) for n in lens) + spare
    width = max(1, max(-(-n // page) for n in lens)) + 1
    table = make_table(rng, lens, page, pages, width)
    k, ks = random_cache(g, pages, H, page, D, kv)
    v, vs = random_cache(g, pages, H, page, D, kv)
    N, Hq = int(starts[-1]) + pad, H * G
    if strided:        # heads and tokens inside a wider projection
        q = rand(g, N, Hq + 3, D + 24, dtype=qt).cuda()[:, 2:2 + Hq, 8:8 + D]
    else:
        q = rand(g, N, Hq, D, dtype=qt).cuda()
    o = torch.full((N, Hq, D), 7.0, dtype=TYPES[qt], device="cuda")
    lse = torch.full((N, Hq), 7.0, dtype=torch.float32, device="cuda")
    i32 = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()
    args = (q, k, v, i32(table), i32(lens), i32(starts))
    wb.kv_attend_chunk(*args, o, scale=scale, window=window, lse=lse, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    worst = check(o, lse, q, stored64(k, ks), stored64(v, vs), table, lens, starts, page,
                  1 / math.sqrt(D) if scale is None else scale, window, kv, qt)
    print(f"[worst] {worst:.3f} of the bound", flush=True)
    assert (o[N - pad:] == 7).all() and (lse[N - pad:] == 7).all()                          # rows of no request
    again = torch.full_like(o, 7.0)
    wb.kv_attend_chunk(*args, again, scale=scale, window=window, k_scale=ks, v_scale=vs)    # without lse
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), o.view(torch.int16))                        # the same bits


NEWS = [1, 0, 5, 31, 32, 33, 64, 65, 130, 3]
PASTS = [0, 9, 0, 1, 31, 64, 63, 200, 0, 700]


@pytest.mark.parametrize("kv,qt", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_types_and_widths(kv, qt, D):
    run(kv, qt, D, 2, 4, NEWS, PASTS, 16, seed=D, pad=3)


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (2, 5), (1, 16), (2, 17), (1, 40), (1, 130), (1, 300)])
def test_head_layouts(H, G):
    run("bf16", "bf16", 64, H, G, [5, 70, 1], [3, 40, 128], 32, seed=G, strided=True)


@pytest.mark.parametrize("page", [8, 16, 64, 256, 4096])
def test_page_sizes(page):
    run("bf16", "bf16", 64, 2, 2, [1, 9, 64, 40, 100], [0, page, page - 1, page + 1, 2 * page + 5], page, seed=page)
    run("e4m3", "bf16", 128, 1, 3, [7, 90], [page - 1, page + 1], page, seed=page + 1)
    run("f16", "f16", 256, 1, 3, [7, 90], [page - 1, page + 1], page, seed=page + 2)


@pytest.mark.parametrize("window", [1, 5, 64, 100, 257, 100000])
def test_window(window):
    run("f16", "f16", 128, 2, 4, [1, 0, 3, 100, 300, 129], [0, 40, 500, 37, 64, 640], 16, window=window, seed=window)
    run("e4m3", "f16", 64, 1, 2, [80, 99], [3, 700], 32, window=window, seed=window + 1)


@pytest.mark.parametrize("kv,qt,D,H,G", [("bf16", "bf16", 128, 2, 4), ("e4m3", "bf16", 128, 1, 8), ("f16", "f16", 256, 2, 8),
                                         ("e4m3", "f16", 64, 3, 1)])
def test_long_caches_are_split_and_joined(kv, qt, D, H, G):
    run(kv, qt, D, H, G, [7], [9000], 64, seed=3)
    run(kv, qt, D, H, G, [1, 40, 0, 200, 3], [5000, 0, 40, 3333, 700], 16, seed=4, pad=5)


@pytest.mark.parametrize("R,most,past,window", [(300, 9, 60, 0), (130, 40, 300, 100), (700, 2, 100, 0)])
def test_batches_past_the_lane_count(R, most, past, window):
    rng = np.random.default_rng(R)
    news, pasts = rng.integers(0, most, R), rng.integers(0, past, R)
    news[-1], pasts[-1] = 4 * most, 8 * past
    run("bf16", "bf16", 64, 2, 2, [int(n) for n in news], [int(n) for n in pasts], 16, window=window, seed=R)


def test_one_prompt():
    run("bf16", "bf16", 128, 2, 4, [1500], [0], 64, seed=8)
    run("f16", "f16", 64, 1, 2, [2049], [1], 128, seed=9)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales(scale):
    run("bf16", "bf16", 128, 1, 4, [1, 50, 100], [5, 0, 300], 16, scale=scale, seed=6)
    run("e4m3", "f16", 128, 1, 4, [1, 50], [5, 300], 16, scale=scale, seed=7)
