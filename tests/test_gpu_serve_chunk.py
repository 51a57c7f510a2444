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


# ---------------------------------------------------------------------------- what rows do not see
def spoiled(c, s, where, kv, D):
    """Infinities and NaN at `where` [pages, page] of a cache, in two columns of three, and NaN scales there."""
    out = where[:, None, :].expand(c.shape[:3]).cuda()
    bad = torch.full_like(c, math.nan, dtype=torch.float32) if kv == "e4m3" else torch.where(
        torch.arange(D, device="cuda") % 3 == 0, math.inf, math.nan).expand(c.shape)
    mix = torch.where(out[..., None] & (torch.arange(D, device="cuda") % 3 != 2), bad, c.float()).to(c.dtype)
    c.view(torch.uint8).copy_(mix.view(torch.uint8))
    if s is not None:
        s.masked_fill_(out, math.nan)


@pytest.mark.parametrize("kv,qt", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 37])
def test_what_is_stored_outside_the_range_leaves_no_trace(kv, qt, D, window):
    """Behind a request's last token, before its windows, in pages of nobody."""
    import linear_attn_decode_amd as wb
    print(f"[case] outside kv={kv} q={qt} D={D} window={window}", flush=True)
    news, pasts, page, H = [1, 13, 45, 100, 0], [0, 0, 63, 411, 30], 16, 2
    lens, starts = [a + b for a, b in zip(news, pasts)], np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    g = torch.Generator().manual_seed(1)
    rng = np.random.default_rng(1)
    pages = sum(-(-n // page) for n in lens) + 2
    table = make_table(rng, lens, page, pages, 40)
    k, ks = random_cache(g, pages, H, page, D, kv)
    v, vs = random_cache(g, pages, H, page, D, kv)
    used = np.zeros((pages, page), bool)
    for r, n in enumerate(lens):
        t = np.arange(max(0, pasts[r] + 1 - window) if window else 0, n)
        used[table[r][t // page], t % page] = True
    clean = [stored64(k, ks), stored64(v, vs)]
    for c, s in ((k, ks), (v, vs)):
        spoiled(c, s, ~torch.from_numpy(used), kv, D)
    q = rand(g, int(starts[-1]), 4, D, dtype=qt).cuda()
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    i32 = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()
    wb.kv_attend_chunk(q, k, v, i32(table), i32(lens), i32(starts), o, window=window, lse=lse, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    check(o, lse, q, *clean, table, lens, starts, page, 1 / math.sqrt(D), window, kv, qt)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("spot", [0, 70, 131, 199])
def test_a_token_that_only_later_rows_see(kv, D, spot):
    """NaN and infinities in the values of one token of a prompt: rows before it are as without it, in
    later ones its columns are NaN and the others as they were."""
    import linear_attn_decode_amd as wb
    print(f"[case] later rows kv={kv} D={D} spot={spot}", flush=True)
    n, page, H, G, window = 200, 16, 2, 3, 90
    qt = "bf16" if kv == "e4m3" else kv
    g = torch.Generator().manual_seed(spot)
    k, ks = random_cache(g, 13, H, page, D, kv)
    v, vs = random_cache(g, 13, H, page, D, kv)
    q = rand(g, n, H * G, D, dtype=qt).cuda()
    table = np.arange(13, dtype=np.int32)[None, ::-1].copy()
    i32 = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    args = (q, k, v, i32(table), i32([n]), i32([0, n]), o)
    clean = [stored64(k, ks), stored64(v, vs)]
    bad = [0, D // 2 - 1, D - 1]
    for h, value in ((0, math.nan), (1, math.nan if kv == "e4m3" else math.inf)):
        row = v[table[0][spot // page], h, spot % page].float()
        row[bad] = value
        v[table[0][spot // page], h, spot % page] = row.to(v.dtype)
    wb.kv_attend_chunk(*args, window=window, lse=lse, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    sees = torch.zeros(n, dtype=torch.bool)
    sees[spot:spot + window] = True
    assert not torch.isfinite(o[sees.cuda()][:, :, bad]).any()
    assert torch.isfinite(o[~sees.cuda()]).all()
    o[:, :, bad] = torch.where(torch.isfinite(o[:, :, bad]), o[:, :, bad], 0)
    ro, _, W, size = O.attend_chunk(q.double().cpu().numpy(), *(c[table[0][np.arange(n) // page], :, np.arange(n) % page] for c in clean),
                                    1 / math.sqrt(D), window)
    ro[np.ix_(sees.numpy(), np.arange(H * G), bad)] = 0
    tol, _ = bounds(kv, qt, D, n, ro, np.zeros((n, H * G)), W, size, np.abs(clean[1]).max())
    assert (np.abs(o.double().cpu().numpy() - ro) <= tol).all()


def test_rows_of_minus_infinity_and_nan_keys():
    import linear_attn_decode_amd as wb
    page, D = 16, 64
    q = torch.ones((30, 2, D), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((6, 1, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    k[0:2] = -math.inf
    k[3, 0, 5, 3] = math.nan                                   # token 21 of the second request, new token 9 of it
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32).cuda()
    lens, starts = torch.tensor([30, 32, 10], dtype=torch.int32).cuda(), torch.tensor([0, 10, 30, 30], dtype=torch.int32).cuda()
    o, lse = torch.empty_like(q), torch.empty((30, 2), device="cuda")
    wb.kv_attend_chunk(q, k, v, table, lens, starts, o, lse=lse)
    torch.cuda.synchronize()
    assert (o[:10] == 0).all() and torch.isneginf(lse[:10]).all()
    assert (o[10:19] == 1).all() and torch.isfinite(lse[10:19]).all()
    assert torch.isnan(o[19:]).all() and torch.isnan(lse[19:]).all()


def test_lowest_values_and_far_apart_scores():
    """Keys at the type's lowest finite value give weights of exactly 0 beside an ordinary one."""
    import linear_attn_decode_amd as wb
    page, D, n = 16, 128, 640
    q = torch.zeros((300, 1, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    k = torch.zeros((40, 1, page, D), dtype=torch.bfloat16, device="cuda")
    k[..., 0] = torch.finfo(torch.bfloat16).min
    v = torch.full_like(k, 3.0)
    k[20, 0, 7, 0] = 1.0
    v[20, 0, 7] = -2.0
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    o, lse = torch.empty_like(q), torch.empty((300, 1), device="cuda")
    wb.kv_attend_chunk(q, k, v, i32([list(range(40))]), i32([n]), i32([0, 300]), o, scale=1.0, lse=lse)
    torch.cuda.synchronize()
    assert (o == -2).all() and (lse - 1.0).abs().max().item() < 1e-6


@pytest.mark.parametrize("gap", [9.0, 15.0, 17.5])
@pytest.mark.parametrize("kv", ["bf16", "f16"])
def test_one_token_far_above_all_others(kv, gap):
    """A token of value 0 that takes nearly all the weight, `gap` above n - 1 equal ones that make up the row."""
    import linear_attn_decode_amd as wb
    page, D, n, m = 64, 128, 20000, 70
    k = torch.zeros((313, 1, page, D), dtype=TYPES[kv], device="cuda")
    v = torch.full_like(k, 64.0)
    k[0, 0, 5, 0] = gap
    v[0, 0, 5] = 0
    q = torch.zeros((m, 1, D), dtype=TYPES[kv], device="cuda")
    q[..., 0] = 1
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    o, lse = torch.empty_like(q), torch.empty((m, 1), device="cuda")
    wb.kv_attend_chunk(q, k, v, i32([list(range(313))]), i32([n]), i32([0, m]), o, scale=1.0, lse=lse)
    torch.cuda.synchronize()
    seen = np.arange(n - m + 1, n + 1)
    rest = (seen - 1) * math.exp(-gap)
    ro = (64.0 * rest / (1 + rest))[:, None]
    half = torch.finfo(TYPES[kv]).eps / 2
    r = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
    A = max(1.0, gap)
    e_s = (D + 8) * U * A + 2.0 ** -22 * A
    tol = ro * (half + (2 * e_s + r + 2 * (96 + n / 16) * U) * (1 + half)) + (2.0 ** -25 + n * 2.0 ** -36 * 64 if kv == "f16" else 0)
    assert (np.abs(o[:, 0].double().cpu().numpy() - ro) <= tol).all()


def test_bad_lengths_pages_and_starts():
    """NaN for the rows of a request whose length is out of range and for those that see a bad page; no rows for
    one whose starts are; everybody else as ever."""
    import linear_attn_decode_amd as wb
    page, D, width = 16, 64, 4
    news = [10, 3, 3, 20, 20, 5, 3, 3, 20, 7]
    lens = [20, -1, 65, 20, 20, 4, -2 ** 31, 2 ** 31 - 1, 20, 64]
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    g = torch.Generator().manual_seed(2)
    k, v = (rand(g, 30, 2, page, D, dtype="f16").cuda() for _ in range(2))
    table = np.arange(len(lens) * width, dtype=np.int32).reshape(len(lens), width) % 30
    table[3, 1], table[4, 0], table[8, 2] = -1, 30, 10 ** 9            # the last is behind the request's tokens
    N = int(starts[-1])
    q = rand(g, N, 4, D, dtype="f16").cuda()
    i32 = lambda a: torch.tensor(np.asarray(a, np.int64).astype(np.int32)).cuda()
    o, lse = torch.empty_like(q), torch.empty((N, 4), device="cuda")
    wb.kv_attend_chunk(q, k, v, i32(table), i32(lens), i32(starts), o, lse=lse)
    torch.cuda.synchronize()
    rows = lambda r: slice(starts[r], starts[r + 1])
    for r in (1, 2, 4, 5, 6, 7):
        assert torch.isnan(o[rows(r)]).all() and torch.isnan(lse[rows(r)]).all(), r
    assert torch.isnan(o[rows(3)][16:]).all()                             # (rows of positions 16 .. 19 see the bad page)
    check(o, lse, q, stored64(k, None), stored64(v, None), table, [n if 0 <= n <= 64 else 0 for n in lens], starts, page,
          1 / math.sqrt(D), 0, "f16", "f16", skip=(1, 2, 3, 4, 5, 6, 7))
    for bad in ([0, -5, 10], [0, 30, 10], [0, 10, N + 1]):
        o.fill_(7)
        wb.kv_attend_chunk(q, k, v, i32(table[:2]), i32([40, 64]), i32(bad), o)
        torch.cuda.synchronize()
        n = 10 if bad[1] == 10 else 30 if bad[1] == 30 else 0
        assert torch.isfinite(o[:n]).all() and (o[:n] != 7).any() if n else True
        assert (o[max(n, 10):] == 7).all() or bad[1] == -5


def test_cache_past_32_bits():
    """Pages whose byte and element offsets pass 2^32."""
    import linear_attn_decode_amd as wb
    page, H, D, pages = 64, 8, 128, 70000             # 4.6e9 elements, 9.2 GB each
    k = torch.zeros((pages, H, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    lens, ids = [100, 64], [[69999, 34000], [65600, 1]]
    g = torch.Generator().manual_seed(3)
    new = [rand(g, 164, H, D, dtype="bf16").cuda() for _ in range(2)]
    slots = [ids[0][t // page] * page + t % page for t in range(100)] + [ids[1][0] * page + t for t in range(64)]
    wb.kv_append(*new, k, v, torch.tensor(slots).cuda())
    q = rand(g, 90, 16, D, dtype="bf16").cuda()
    starts = np.array([0, 30, 90], np.int32)
    i32 = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()
    o, lse = torch.empty_like(q), torch.empty((90, 16), device="cuda")
    wb.kv_attend_chunk(q, k, v, i32(ids), i32(lens), i32(starts), o, lse=lse)
    torch.cuda.synchronize()
    for r, rows in enumerate((slice(0, 100), slice(100, 164))):
        kk, vv = (x[rows].double().cpu().numpy().transpose(1, 0, 2)[None] for x in new)
        at = slice(starts[r], starts[r + 1])
        check(o[at], lse[at], q[at], kk, vv, np.zeros((1, 1), np.int32), [lens[r]], [0, starts[r + 1] - starts[r]], 4096,
              1 / math.sqrt(D), 0, "bf16", "bf16")


def test_no_tokens():
    import linear_attn_decode_amd as wb
    k = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    wb.kv_attend_chunk(q, k, k.clone(), i32([[0]]), i32([0]), i32([0, 0]), torch.empty_like(q))
    torch.cuda.synchronize()


def test_single_tokens_agree_with_kv_attend():
    """A batch of one new token each: the two operators under their bounds of one another."""
    import linear_attn_decode_amd as wb
    g = torch.Generator().manual_seed(4)
    page, H, D, R = 16, 2, 128, 9
    lens = [1, 5, 64, 65, 300, 700, 1000, 2, 128]
    k, v = (rand(g, 200, H, page, D, dtype="bf16").cuda() for _ in range(2))
    table = torch.from_numpy(make_table(np.random.default_rng(0), lens, page, 200, 70)).cuda()
    q = rand(g, R, 8, D, dtype="bf16").cuda()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    one, many = torch.empty_like(q), torch.empty_like(q)
    l1, l2 = torch.empty((R, 8), device="cuda"), torch.empty((R, 8), device="cuda")
    wb.kv_attend(q, k, v, table, i32(lens), one, lse=l1)
    wb.kv_attend_chunk(q, k, v, table, i32(lens), i32(list(range(R + 1))), many, lse=l2)
    torch.cuda.synchronize()
    assert (l1 - l2).abs().max().item() < 1e-4
    assert (one.float() - many.float()).abs().max().item() < 4 * 2.0 ** -8 * v.float().abs().max().item()
