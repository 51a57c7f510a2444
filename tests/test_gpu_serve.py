"""GPU parity of the serving operators (include/wbserve.h) with their float64 definitions
(oracle/serving.py).

Tolerances, from the arithmetic (u = 2^-24, half a float32 step):
  * attention: a score is a float32 sum of D exact products, scaled once or twice: within
    (D + 4) u sum|scale q k|; a weight e^{s - m} adds the rounding of s - m and of the
    exponential, 2^-22 together, relative to max(1, |s|). The sums over tokens take 32 products a step and then a step
    per tile: (32 + n / 32 + 64) u of sum p|v|; the weights' two 16-bit limbs leave 2^-17 of
    a weight; the output is rounded once (half a step of its type). So
      |o - o*| <= eps/2 |o*| + W (2 e_s + 2^-17 + 2 (96 + n/32) u),  W = sum p|v| / sum p,
      |lse - lse*| <= e_s + (96 + n/32) u + 2 u |lse*|,  e_s = (D + 4) u A + 2^-22 max(1, A),
    A the largest sum|scale q k|. The limbs of a float16 cache also leave the smallest float16
    step, 2^-25 of a weight of 1 (and 2^-25 of the values' size per token): n 2^-25 max|v|.
  * e4m3: scale within 2 u of max|x| / 448; code * scale within half a step of x (the
    quotient's own rounding moves a tie by 2 u).
  * norm: the float32 sum of D squares is D / 256 + 16 additions deep at most in any of the
    kernels (one row: 256 lanes or more, or at most 64 values a lane), and y takes 8 more
    roundings: relative (D / 256 + 64 + 24) u of y.
Integers (planning) are equal.
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
    """Every request's pages from a shuffled pool; entries behind a request's last are ids
    of nobody (they must not be read)."""
    order = rng.permutation(pages)
    table = np.full((len(lens), width), 1 << 30, np.int32)
    at = 0
    for r, n in enumerate(lens):
        c = -(-n // page)
        table[r, :c] = order[at:at + c]
        at += c
    return table


def check_attend(o, lse, q, k, v, table, lens, page, scale, window, skip=()):
    eps = torch.finfo(o.dtype).eps
    o, lse, q = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    f16 = eps < 2.0 ** -8
    worst = 0.0
    for r, n in enumerate(lens):
        if r in skip:
            continue
        t = np.arange(n)
        at = table[r][t // page]
        kr, vr = k[at, :, t % page], v[at, :, t % page]
        ro, rl, W, size = O.attend(q[r], kr, vr, scale, window)
        A = max(1.0, size.max())
        e_s = (q.shape[2] + 4) * U * A + 2.0 ** -22 * A
        sums = (96 + n / 32) * U
        tol = eps / 2 * np.abs(ro) + W * (2 * e_s + 2.0 ** -17 + 2 * sums) + 2.0 ** -40
        if f16:
            tol += n * 2.0 ** -25 * (np.abs(vr).max() if n else 0)
        err = np.abs(o[r] - ro)
        assert (err <= tol).all(), (r, n, float((err / tol).max()))
        worst = max(worst, float((err / tol).max()))
        both = np.isneginf(rl)
        assert (np.isneginf(lse[r]) == both).all(), (r, n)
        ltol = e_s + sums + 2 * U * np.abs(rl[~both])
        assert (np.abs(lse[r][~both] - rl[~both]) <= ltol).all(), (r, n)
    return worst


def run_attend(kv, qt, D, H, G, lens, page, window=0, seed=0, strided=False, scale=None, spare=2):
    import linear_attn_decode_amd as wb
    print(f"[case] attend kv={kv} q={qt} D={D} H={H} G={G} lens={lens[:8]} R={len(lens)} page={page} window={window}", flush=True)
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    pages = sum(-(-n // page) for n in lens) + spare
    width = max(1, max(-(-n // page) for n in lens)) + 1
    table = make_table(rng, lens, page, pages, width)
    k, ks = random_cache(g, pages, H, page, D, kv)
    v, vs = random_cache(g, pages, H, page, D, kv)
    R, Hq = len(lens), H * G
    if strided:        # heads and requests inside a wider projection
        q = rand(g, R, Hq + 3, D + 24, dtype=qt).cuda()[:, 2:2 + Hq, 8:8 + D]
    else:
        q = rand(g, R, Hq, D, dtype=qt).cuda()
    o = torch.full((R, Hq, D), 7.0, dtype=TYPES[qt], device="cuda")
    lse = torch.full((R, Hq), 7.0, dtype=torch.float32, device="cuda")
    args = (q, k, v, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), o)
    wb.kv_attend(*args, scale=scale, window=window, lse=lse, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    worst = check_attend(o, lse, q, stored64(k, ks), stored64(v, vs), table, lens, page,
                         1 / math.sqrt(D) if scale is None else scale, window)
    print(f"[worst] {worst:.3f} of the bound", flush=True)
    again = torch.empty_like(o)
    wb.kv_attend(*args[:5], again, scale=scale, window=window, k_scale=ks, v_scale=vs)      # without lse
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), o.view(torch.int16))                        # the same bits


LENS = [1, 0, 7, 8, 9, 31, 32, 33, 127, 128, 129, 300]


@pytest.mark.parametrize("kv,qt", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_types_and_widths(kv, qt, D):
    run_attend(kv, qt, D, 2, 4, LENS, 16, seed=D)


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (2, 5), (1, 16), (2, 17), (1, 40)])
def test_attend_head_layouts(H, G):
    run_attend("bf16", "bf16", 128, H, G, [5, 64, 200], 32, seed=G, strided=True)


@pytest.mark.parametrize("page", [8, 16, 64, 256, 4096])
def test_attend_page_sizes(page):
    run_attend("bf16", "bf16", 64, 2, 2, [1, page - 1, page, page + 1, 2 * page + 5], page, seed=page)
    run_attend("e4m3", "bf16", 64, 1, 3, [page - 1, page + 1], page, seed=page + 1)


@pytest.mark.parametrize("window", [1, 5, 32, 100, 257, 100000])
def test_attend_window(window):
    run_attend("f16", "f16", 128, 2, 4, [0, 1, 5, 31, 32, 33, 100, 101, 640, 1000], 16, window=window, seed=window)
    run_attend("e4m3", "f16", 64, 1, 2, [3, 99, 700], 32, window=window, seed=window + 1)


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("e4m3", 128), ("f16", 256)])
def test_attend_long_requests_are_split_and_joined(kv, D):
    run_attend(kv, "bf16" if kv == "e4m3" else kv, D, 2, 8, [20011], 64, seed=3)
    run_attend(kv, "bf16" if kv == "e4m3" else kv, D, 1, 4, [1, 9000, 0, 40, 3333], 16, seed=4)


def test_attend_many_requests():
    rng = np.random.default_rng(0)
    run_attend("bf16", "bf16", 64, 1, 2, [int(n) for n in rng.integers(0, 400, 700)], 32, seed=5)


@pytest.mark.parametrize("kv,D,H,G,R,longest,window", [("bf16", 128, 3, 2, 300, 200, 0), ("f16", 64, 2, 1, 1030, 70, 0),
                                                       ("e4m3", 128, 5, 4, 130, 600, 0), ("e4m3", 256, 2, 2, 65, 300, 100),
                                                       ("bf16", 256, 4, 8, 64, 500, 0), ("bf16", 64, 1, 1, 4100, 40, 0)])
def test_attend_batches_past_the_lane_count(kv, D, H, G, R, longest, window):
    """More requests than lanes, idle ones among them, one long one behind many short ones."""
    rng = np.random.default_rng(R)
    lens = [int(n) for n in rng.integers(0, longest, R)]
    lens[R // 3: R // 3 + 5] = [0] * 5
    lens[-1] = 4 * longest
    run_attend(kv, "bf16" if kv == "e4m3" else kv, D, H, G, lens, 16, window=window, seed=R)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attend_scales(scale):
    run_attend("bf16", "bf16", 128, 1, 4, [1, 50, 400], 16, scale=scale, seed=6)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attend_ignores_what_is_stored_outside_the_range(kv):
    """NaN and infinities behind a request's last token, before its window and in pages of
    nobody leave no trace."""
    import linear_attn_decode_amd as wb
    lens, page, window, D, H = [0, 1, 13, 45, 200, 511], 16, 37, 128, 2
    g = torch.Generator().manual_seed(1)
    rng = np.random.default_rng(1)
    pages = sum(-(-n // page) for n in lens) + 2
    table = make_table(rng, lens, page, pages, 40)
    k, ks = random_cache(g, pages, H, page, D, kv)
    v, vs = random_cache(g, pages, H, page, D, kv)
    used = np.zeros((pages, page), bool)
    for r, n in enumerate(lens):
        t = np.arange(max(0, n - window), n)
        used[table[r][t // page], t % page] = True
    out = ~torch.from_numpy(used)[:, None, :].expand(pages, H, page).cuda()
    clean = [stored64(k, ks), stored64(v, vs)]
    for c, s in ((k, ks), (v, vs)):
        bad = torch.full_like(c, math.nan) if kv == "e4m3" else torch.where(torch.arange(D, device="cuda") % 3 == 0, math.inf, math.nan)
        c.view(torch.uint8 if kv == "e4m3" else torch.int16).copy_(
            torch.where(out[..., None], bad.to(c.dtype).float(), c.float()).to(c.dtype).view(torch.uint8 if kv == "e4m3" else torch.int16))
        if s is not None:
            s.masked_fill_(out, math.nan)
    q = rand(g, len(lens), 4, D, dtype="bf16").cuda()
    o, lse = torch.empty_like(q), torch.empty((len(lens), 4), device="cuda")
    wb.kv_attend(q, k, v, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), o, window=window,
                 lse=lse, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    check_attend(o, lse, q, *clean, table, lens, page, 1 / math.sqrt(D), window)


def test_attend_rows_of_minus_infinity_and_nan():
    """Scores that are all -inf leave nothing; a NaN in the range makes the request's rows NaN
    and no other's."""
    import linear_attn_decode_amd as wb
    page, D = 16, 64
    q = torch.ones((3, 2, D), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((6, 1, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    k[0:2] = -math.inf
    k[3, 0, 5, 3] = math.nan
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32).cuda()
    lens = torch.tensor([30, 32, 20], dtype=torch.int32).cuda()
    o, lse = torch.empty_like(q), torch.empty((3, 2), device="cuda")
    wb.kv_attend(q, k, v, table, lens, o, lse=lse)
    torch.cuda.synchronize()
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
    assert (o[2] == 1).all() and torch.allclose(lse[2], torch.full_like(lse[2], math.log(20)), rtol=0, atol=1e-6)


def test_attend_lowest_values_and_far_apart_scores():
    """Keys at the type's lowest finite value give weights of exactly 0 beside an ordinary one."""
    import linear_attn_decode_amd as wb
    page, D = 16, 128
    q = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1
    k = torch.zeros((40, 1, page, D), dtype=torch.bfloat16, device="cuda")
    k[..., 0] = torch.finfo(torch.bfloat16).min
    v = torch.full_like(k, 3.0)
    k[20, 0, 7, 0] = 1.0
    v[20, 0, 7] = -2.0
    table = torch.arange(40, dtype=torch.int32).view(1, 40).cuda()
    o, lse = torch.empty_like(q), torch.empty((1, 1), device="cuda")
    wb.kv_attend(q, k, v, table, torch.tensor([640], dtype=torch.int32).cuda(), o, scale=1.0, lse=lse)
    torch.cuda.synchronize()
    assert (o == -2).all() and abs(float(lse) - 1.0) < 1e-6


def test_attend_bad_lengths_and_pages_are_nan_for_their_request_only():
    import linear_attn_decode_amd as wb
    page, D, width = 16, 64, 4
    lens = [20, -1, 65, 20, 20, 64, -2 ** 31, 2 ** 31 - 1, 20]
    g = torch.Generator().manual_seed(2)
    k, v = (rand(g, 30, 2, page, D, dtype="f16").cuda() for _ in range(2))
    table = np.arange(len(lens) * width, dtype=np.int32).reshape(len(lens), width) % 30
    table[3, 1], table[4, 0], table[8, 2] = -1, 30, 10 ** 9            # the last is behind the request's tokens
    q = rand(g, len(lens), 4, D, dtype="f16").cuda()
    o, lse = torch.empty_like(q), torch.empty((len(lens), 4), device="cuda")
    wb.kv_attend(q, k, v, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), o, lse=lse)
    torch.cuda.synchronize()
    bad = [1, 2, 3, 4, 6, 7]
    assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
    check_attend(o, lse, q, stored64(k, None), stored64(v, None), table, [n if 0 <= n <= 64 else 0 for n in lens], page,
                 1 / math.sqrt(D), 0, skip=bad)


def test_attend_cache_past_32_bits():
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
    q = rand(g, 2, 16, D, dtype="bf16").cuda()
    o, lse = torch.empty_like(q), torch.empty((2, 16), device="cuda")
    wb.kv_attend(q, k, v, torch.tensor(ids, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), o, lse=lse)
    torch.cuda.synchronize()
    assert int(torch.count_nonzero(k[69999, :, :, 0])) > 0
    ro = [x.double().cpu().numpy() for x in new]
    at = {0: slice(0, 100), 1: slice(100, 164)}
    for r in range(2):
        table = np.zeros((1, 1), np.int32)
        kk, vv = (x[at[r]].transpose(1, 0, 2)[None] for x in ro)
        check_attend(o[r:r + 1], lse[r:r + 1], q[r:r + 1], kk, vv, table, [lens[r]], 4096, 1 / math.sqrt(D), 0)


# ---------------------------------------------------------------------------- planning
def run_plan(lens, more, page, width, free_size, n_free, n_slots, seed=0, in_place=False):
    import linear_attn_decode_amd as wb
    print(f"[case] plan R={len(lens)} page={page} width={width} free={n_free}/{free_size} slots={n_slots} in_place={in_place}", flush=True)
    rng = np.random.default_rng(seed)
    R = len(lens)
    table = rng.integers(0, 10000, (R, width)).astype(np.int32)
    free = rng.permutation(free_size + 100)[:free_size].astype(np.int32)
    want = O.plan(lens, more, table, free, n_free, page, n_slots)
    i32 = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()
    dl, dm, dt, df, dn = i32(lens), i32(more), i32(table), i32(free), i32([n_free])
    slots, starts, status = torch.full((n_slots + 2,), 77, dtype=torch.int64, device="cuda")[:n_slots], i32([9] * (R + 1)), i32([9])
    lo, no = (dl, dn) if in_place else (i32([9] * R), i32([9]))
    for _ in range(1 if in_place else 2):                          # (out of place: a second call gives the same)
        wb.plan_pages(dl, dm, dt, df, dn, page, slots, starts, status, lens_out=lo, n_free_out=no)
    torch.cuda.synchronize()
    got = (dt, slots, starts, lo, no, status)
    for name, a, b in zip(("table", "slots", "starts", "lens", "n_free", "status"), got, want):
        assert np.array_equal(a.cpu().numpy().reshape(np.shape(b)), b), name
    assert np.array_equal(df.cpu().numpy(), free)
    return want[5]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,longest,most,page", [(1, 0, 1, 16), (5, 40, 1, 8), (64, 300, 1, 16), (300, 100, 20, 32),
                                                 (256, 50, 200, 16), (1024, 64, 4, 64), (1500, 64, 1, 16), (3000, 33, 40, 8)])
def test_plan(R, longest, most, page, in_place):
    rng = np.random.default_rng(R)
    lens, more = rng.integers(0, longest + 1, R), rng.integers(0, most + 1, R)
    total = int(more.sum())
    for slots in (total, total + 5, max(1, total + 700)):
        assert run_plan(lens, more, page, (longest + most) // page + 2, total + R + 3, total + R, slots, seed=R, in_place=in_place) == 0


def test_plan_that_cannot_be_carried_out_changes_nothing():
    for R, more, slots in ((3, 10, 30), (600, 10, 6000)):              # one launch, two launches
        lens, m = [9] * R, [more] * R
        need = R * (-(-(9 + more) // 8) - 2)
        for in_place in (False, True):
            kw = dict(page=8, seed=1, in_place=in_place)
            assert run_plan(lens, m, width=4, free_size=need + 3, n_free=need, n_slots=slots, **kw) == 0
            assert run_plan(lens, m, width=4, free_size=need + 3, n_free=need - 1, n_slots=slots, **kw) == 4
            assert run_plan(lens, m, width=4, free_size=need + 3, n_free=need + 4, n_slots=slots, **kw) == 1
            assert run_plan(lens, m, width=4, free_size=need + 3, n_free=-1, n_slots=slots, **kw) == 1
            assert run_plan(lens, m, width=2, free_size=need + 3, n_free=need, n_slots=slots, **kw) == 2
            assert run_plan(lens, m, width=4, free_size=need + 3, n_free=need, n_slots=slots - 1, **kw) == 3
            assert run_plan([-1] + lens[1:], m, width=4, free_size=need + 3, n_free=need, n_slots=slots, **kw) == 1
            assert run_plan(lens, m[1:] + [-5], width=4, free_size=need + 3, n_free=need, n_slots=slots, **kw) == 1
    assert run_plan([0, 0], [0, 0], 16, 1, 0, 0, 0) == 0               # nothing at all


@pytest.mark.parametrize("R", [1, 7, 64, 1500])
def test_release(R):
    import linear_attn_decode_amd as wb
    rng = np.random.default_rng(R)
    page, width = 16, 6
    lens, ended = rng.integers(0, width * page + 1, R), rng.integers(0, 2, R)
    table = rng.integers(0, 10000, (R, width)).astype(np.int32)
    held = int(sum(-(-lens // page) * ended))
    i32 = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()
    for size, n_free, bad in ((held + 9, 7, {}), (held + 6, 7, {}), (held + 9, held + 10, {}), (held + 9, 7, {0: -3}), (held + 9, 7, {R - 1: 1000})):
        n = lens.copy()
        for r, x in bad.items():
            n[r] = x
        free = rng.integers(0, 10000, size).astype(np.int32)
        want = O.release(ended, n, table, free, n_free, page)
        dl, df, dn, st = i32(n), i32(free), i32([n_free]), i32([9])
        wb.release_pages(torch.tensor(ended, dtype=torch.uint8).cuda().bool(), dl, i32(table), df, dn, page, st)
        torch.cuda.synchronize()
        for name, a, b in zip(("lens", "free", "n_free", "status"), (dl, df, dn, st), want):
            assert np.array_equal(a.cpu().numpy().reshape(np.shape(b)), b), (name, size, n_free, bad)


# ---------------------------------------------------------------------------- cache writes
@pytest.mark.parametrize("kv,src", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32"), ("e4m3", "bf16"),
                                    ("e4m3", "f16"), ("e4m3", "f32")])
@pytest.mark.parametrize("N,H,D,page,slack", [(1, 1, 64, 8, 0), (37, 3, 128, 16, 64), (200, 2, 256, 64, 8)])
def test_append(kv, src, N, H, D, page, slack):
    import linear_attn_decode_amd as wb
    print(f"[case] append kv={kv} src={src} N={N} H={H} D={D} page={page}", flush=True)
    g = torch.Generator().manual_seed(N)
    rng = np.random.default_rng(N)
    pages = -(-N // page) + 2
    rows = rand(g, N, 2 * H * D + slack, dtype="f32")
    rows *= torch.exp(3 * torch.randn((N, 1), generator=g))
    rows[N // 2] = 0                                                     # a vector of zeros
    rows = rows.to(TYPES[src]).cuda()
    k, v = rows[:, :H * D].unflatten(1, (H, D)), rows[:, H * D + slack:].unflatten(1, (H, D))
    kc, ks = random_cache(g, pages, H, page, D, kv)
    vc, vs = random_cache(g, pages, H, page, D, kv)
    before = [t if t is None else t.clone() for t in (kc, vc, ks, vs)]
    slots = rng.permutation(pages * page)[:N].astype(np.int64)
    slots[::5] = -1                                                      # padding
    if N > 10:
        slots[1], slots[2], slots[3] = pages * page, -2 ** 62, 2 ** 62   # outside
    wb.kv_append(k, v, kc, vc, torch.from_numpy(slots).cuda(), k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    keep = (slots >= 0) & (slots < pages * page)
    at, off = slots[keep] // page, slots[keep] % page
    for x, cache, scale, old, old_scale in ((k, kc, ks, before[0], before[2]), (v, vc, vs, before[1], before[3])):
        raw = torch.uint8 if kv == "e4m3" else torch.int16
        untouched = np.ones((pages, page), bool)
        untouched[at, off] = False
        same = (cache.view(raw) == old.view(raw)).all(3).cpu().numpy().transpose(0, 2, 1)
        assert same[untouched].all()
        x64 = x.double().cpu().numpy()[keep]
        got = cache[torch.from_numpy(at).cuda(), :, torch.from_numpy(off).cuda()]
        if kv != "e4m3":
            assert torch.equal(got, x[torch.from_numpy(keep).cuda()].to(TYPES[kv]))
            continue
        assert (scale == old_scale).cpu().numpy().transpose(0, 2, 1)[untouched].all()
        sc = scale.double().cpu().numpy()[at, :, off]
        want = O.group_scale(x64)
        assert (np.abs(sc - want) <= 2 * U * want).all()
        q = x64 / np.where(sc > 0, sc, 1.0)[..., None]
        err = np.abs(got.double().cpu().numpy() - q)
        assert (err <= O.e4m3_half_step(q) + 2 * U * np.abs(q)).all()
        assert (got.float()[torch.from_numpy(want == 0).cuda()] == 0).all()


def test_append_non_finite_and_tiny_vectors():
    import linear_attn_decode_amd as wb
    D, page = 64, 8
    k = torch.ones((5, 1, D))
    k[0, 0, 3], k[1, 0, 5], k[2], k[3] = math.nan, -math.inf, 1e-37, 0.0
    k[4] = torch.linspace(-1, 1, D) * 2.0 ** -120
    kc = torch.zeros((1, 1, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    vc, ks = torch.zeros_like(kc), torch.zeros((1, 1, page), device="cuda")
    vs = torch.zeros_like(ks)
    wb.kv_append(k.cuda(), k.cuda(), kc, vc, torch.arange(5).cuda(), k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    for c, s in ((kc, ks), (vc, vs)):
        back = (c.float() * s[..., None])[0, 0].cpu()
        assert torch.isnan(back[:2]).all() and (back[3] == 0).all()
        assert torch.isfinite(back[2:]).all() and float(s[0, 0, 2]) == 2.0 ** -126
        assert (back[2] - 1e-37).abs().max() <= 2.0 ** -126 * 2 ** -4 * 8 + 1e-45      # half a step of 8.5 below 16
        assert (back[4] - k[4, 0]).abs().max() <= 2.0 ** -120 * 2 ** -4


# ---------------------------------------------------------------------------- norm
def run_norm(N, D, dt, residual, group, slack=0, weight=True, in_place=False, seed=0, eps=1e-6, shift=0):
    import linear_attn_decode_amd as wb
    print(f"[case] norm N={N} D={D} {dt} residual={residual} group={group} slack={slack} weight={weight}", flush=True)
    g = torch.Generator().manual_seed(seed + D)
    spread = torch.exp(2 * torch.randn((N, 1), generator=g))

    def rows():
        return (rand(g, N, D + slack) * spread).to(TYPES[dt]).cuda()[:, shift:shift + D]
    x = rows()
    r = rows() if residual else None
    w = (1 + 0.3 * rand(g, D)).to(TYPES[dt]).cuda() if weight else None
    r64 = None if r is None else r.double().cpu().numpy()
    out = r if in_place else (rows() if residual else None)
    cw = torch.zeros((N, D + slack), dtype=torch.uint8, device="cuda")
    codes = cw.view(torch.float8_e4m3fn)[:, shift:shift + D]
    scales = torch.empty((N, -(-D // group) if group else 1), device="cuda")
    wb.norm_quant(x, w, codes, scales, eps=eps, group=group, residual=r, residual_out=None if in_place else out)
    torch.cuda.synchronize()
    x64 = x.double().cpu().numpy()
    h, y, want = O.norm(x64, r64, None if w is None else w.double().cpu().numpy(), eps, group)
    rel = (D / 256 + 64 + 24) * U
    # (h is a float32 sum: its rounding is relative to h, which is what the norm takes)
    sc = scales.double().cpu().numpy()
    assert (np.abs(sc - want) <= (rel + 2 * U) * want).all()
    q = y / np.repeat(np.where(sc > 0, sc, 1.0), group or D, axis=1)[:, :D]
    err = np.abs(codes.double().cpu().numpy() - np.clip(q, -448, 448))
    tol = O.e4m3_half_step(np.clip(q, -448, 448)) + 2 * rel * np.abs(q)
    assert (err <= tol).all(), float((err / tol).max())
    if residual:
        t = torch.finfo(TYPES[dt]).eps
        assert (np.abs(out.double().cpu().numpy() - h) <= t / 2 * np.abs(h) * (1 + 2 * U) + U * np.abs(h)).all()
    if slack:                                                            # between the rows: left as it was
        rest = cw.clone()
        rest[:, shift:shift + D] = 0
        assert not rest.any()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [1, 7, 8, 127, 128, 129, 256, 1000, 1024, 2048, 4097, 5000, 8192, 16384])
def test_norm_widths(dt, D):
    run_norm(3, D, dt, True, 128, seed=1)
    run_norm(5, D, dt, False, 0, seed=2)


@pytest.mark.parametrize("D", [128, 640, 1032, 4096])
@pytest.mark.parametrize("slack,shift", [(8, 0), (5, 0), (16, 1)])
def test_norm_strides_and_alignment(D, slack, shift):
    run_norm(9, D, "bf16", True, 128, slack=slack, shift=shift)
    run_norm(6, D, "f32", True, 0, slack=slack, shift=shift, in_place=True)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("base", [0, 56, 120, 248, 1040])
def test_norm_row_ends(dt, base):
    """Every length of a row's last chunk, at each number of lanes a row takes."""
    for tail in range(1, 8):
        run_norm(37, base + tail, dt, True, 128, slack=3, shift=1, seed=tail)
        run_norm(37, base + tail, dt, False, 0, seed=tail)


@pytest.mark.parametrize("N", [1, 2, 63, 64, 1023, 5000])
def test_norm_rows(N):
    run_norm(N, 128, "f32", False, 0, seed=N)
    run_norm(N, 200, "bf16", True, 128, seed=N, in_place=True, weight=False)


def test_norm_widest_rows():
    run_norm(2, 65536, "bf16", True, 128)
    run_norm(2, 65535, "f32", False, 0)


@pytest.mark.parametrize("log2w", [-140, -126, -122, -119, -118, -100, 0, 100, 124])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_scales_at_the_ends_of_the_range(log2w, group):
    """Weights that put a scale at its least value, beside it, and a row's values near the
    largest float32. (Products below the normal numbers are off by 2^-150 each: 2^-22 of a
    scale, two of them.)"""
    import linear_attn_decode_amd as wb
    N, D = 64, 200
    g = torch.Generator().manual_seed(200 + log2w)
    x = rand(g, N, D) * torch.exp(2 * torch.randn((N, 1), generator=g))
    w = torch.ldexp(1 + 0.3 * torch.rand(D, generator=g), torch.tensor(log2w))
    codes = torch.empty((N, D), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((N, -(-D // group) if group else 1), device="cuda")
    wb.norm_quant(x.cuda(), w.cuda(), codes, scales, eps=1e-6, group=group)
    torch.cuda.synchronize()
    _, y, want = O.norm(x.double().numpy(), None, w.double().numpy(), 1e-6, group)
    rel = (D / 256 + 64 + 24) * U
    sc = scales.double().cpu().numpy()
    assert (np.abs(sc - want) <= (rel + 2 * U) * want).all()
    q = np.clip(y / np.repeat(sc, group or D, axis=1)[:, :D], -448, 448)
    err = np.abs(codes.double().cpu().numpy() - q)
    assert (err <= O.e4m3_half_step(q) + 2 * rel * np.abs(q) + 2.0 ** -21).all()


def test_norm_zero_and_non_finite_rows():
    import linear_attn_decode_amd as wb
    x = torch.ones((4, 512), device="cuda")
    x[0] = 0
    x[1, 200] = math.nan
    x[2, 300] = math.inf
    x[3, 128:256] = 0                                                    # a group of zeros
    codes, scales = torch.empty((4, 512), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((4, 4), device="cuda")
    wb.norm_quant(x, None, codes, scales, eps=0.0, group=128)
    torch.cuda.synchronize()
    c = codes.float()
    assert torch.isnan(c[1]).all() and torch.isnan(c[2, 300])
    assert (c[3, 128:256] == 0).all() and float(scales[3, 1]) == 0 and (c[3, :128] == 448).all()
    wb.norm_quant(x[:1], None, codes[:1], scales[:1], eps=1e-6, group=128)
    torch.cuda.synchronize()
    assert (codes[0].float() == 0).all() and (scales[0] == 0).all()


def test_empty_calls():
    import linear_attn_decode_amd as wb
    z = torch.empty((0, 64), device="cuda")
    wb.norm_quant(z, None, z.to(torch.float8_e4m3fn), torch.empty((0, 1), device="cuda"))
    kc = torch.zeros((1, 1, 8, 64), dtype=torch.bfloat16, device="cuda")
    n = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    wb.kv_append(n, n, kc, kc.clone(), torch.empty(0, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------- together
def serving_loop(kv, stream=None):
    """Prompts of several requests, then decode steps: plan, append, attend, with requests
    that end and are replaced; every step against the oracle on what is stored."""
    import linear_attn_decode_amd as wb
    R, H, G, D, page, width, pages = 5, 2, 4, 64, 16, 6, 24
    g = torch.Generator().manual_seed(11)
    rng = np.random.default_rng(11)
    dt = torch.bfloat16
    shape = (pages, H, page, D)
    kc, vc = (torch.zeros(shape, dtype=TYPES[kv], device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(shape[:3], device="cuda") if kv == "e4m3" else None for _ in range(2))
    lens, n_free, status = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (R, 1, 1))
    free = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()
    n_free.fill_(pages)
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    starts = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
    history = [[] for _ in range(R)]                       # (k, v) of every token, as given
    for step in range(30):
        if step == 0:
            more = [20, 0, 33, 1, 7]
        elif step % 7 == 3:                                # a request ends, another takes its place
            r = step // 7 % R
            history[r] = []
            ended = torch.zeros(R, dtype=torch.bool)
            ended[r] = True
            wb.release_pages(ended.cuda(), lens, table, free, n_free, page, status)
            more = [1] * R
            more[r] = 18
        else:
            more = [1, step % 2, 1, 1, 1]
        total = sum(more)
        slots = torch.empty(total + 3, dtype=torch.int64, device="cuda")       # padded batch
        wb.plan_pages(lens, torch.tensor(more, dtype=torch.int32).cuda(), table, free, n_free, page, slots, starts, status)
        k, v = (rand(g, total + 3, H, D).to(dt).cuda() for _ in range(2))
        wb.kv_append(k, v, kc, vc, slots, k_scale=ks, v_scale=vs)
        q = rand(g, R, H * G, D).to(dt).cuda()
        o, lse = torch.empty_like(q), torch.empty((R, H * G), device="cuda")
        wb.kv_attend(q, kc, vc, table, lens, o, lse=lse, k_scale=ks, v_scale=vs)
        torch.cuda.synchronize()
        assert int(status) == 0
        at = 0
        for r, m in enumerate(more):
            for i in range(m):
                history[r].append((k[at + i], v[at + i]))
            at += m
        n = lens.cpu().tolist()
        assert n == [len(x) for x in history]
        assert int(n_free) == pages - sum(-(-x // page) for x in n)
        t = table.cpu().numpy()
        k64, v64 = stored64(kc, ks), stored64(vc, vs)
        check_attend(o, lse, q, k64, v64, t, n, page, 1 / math.sqrt(D), 0)
        for r in range(R):                                  # what is stored is what was given
            i = np.arange(n[r])
            for which, stored in ((0, k64), (1, v64)):
                if n[r]:
                    given = torch.stack([x[which] for x in history[r]]).double().cpu().numpy()
                    err = np.abs(stored[t[r][i // page], :, i % page] - given)
                    assert err.max() <= (np.abs(given).max() / 16 if kv == "e4m3" else 0.0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_plan_append_attend_together(kv):
    print(f"[case] serving loop {kv}", flush=True)
    serving_loop(kv)


def test_readout_into_the_norm():
    """The float32 readout of a write-back decode step goes into the norm as it is."""
    import linear_attn_decode_amd as wb
    from synth import decode_inputs
    B, H, d = 2, 3, 128
    st = wb.WriteBackState("had_int8", "rtn", B, H, d, d, True, block=128)
    inp = {n: torch.from_numpy(a).cuda() for n, a in decode_inputs(1, B, H, d, d, 2).items()}
    o = torch.zeros((B, H, d), device="cuda")
    codes, scales = torch.empty((B * H, d), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((B * H, 1), device="cuda")
    w = torch.rand(d, device="cuda") + 0.5
    for t in range(2):
        st.step_decode(inp["q"][t], inp["k"][t], inp["v"][t], inp["beta"][t], inp["s"], o, t)
        wb.norm_quant(o.view(B * H, d), w, codes, scales)
    torch.cuda.synchronize()
    _, y, want = O.norm(o.view(B * H, d).double().cpu().numpy(), None, w.double().cpu().numpy(), 1e-6, 0)
    rel = (d / 256 + 88) * U
    sc = scales.double().cpu().numpy()
    assert (np.abs(sc - want) <= (rel + 2 * U) * want).all()
    q = np.clip(y / sc, -448, 448)
    assert (np.abs(codes.double().cpu().numpy() - q) <= O.e4m3_half_step(q) + 2 * rel * np.abs(q)).all()


def test_captured_step_replays_with_changing_inputs():
    """One decode step (plan in place, append, attend, norm) captured once; every replay
    against the same calls made eagerly from the same state, with eager work between."""
    import linear_attn_decode_amd as wb
    R, H, G, D, page, width, pages = 4, 2, 4, 128, 16, 40, 200

    def fresh():
        g = torch.Generator().manual_seed(21)
        s = dict(kc=torch.zeros((pages, H, page, D), dtype=torch.bfloat16, device="cuda"))
        s["vc"] = torch.zeros_like(s["kc"])
        s["free"] = torch.randperm(pages, generator=g).int().cuda()
        s["n_free"] = torch.tensor([pages], dtype=torch.int32).cuda()
        s["lens"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        s["table"] = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
        s["starts"], s["status"] = torch.zeros(R + 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.zeros(64 * R, dtype=torch.int64, device="cuda")
        s["more"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        s["k"], s["v"] = (torch.zeros((64 * R, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        s["q"] = torch.zeros((R, H * G, D), dtype=torch.bfloat16, device="cuda")
        s["o"] = torch.zeros_like(s["q"])
        s["codes"] = torch.zeros((R, H * G * D), dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.zeros((R, H * G * D // 128), device="cuda")
        return s

    def step(s):
        wb.plan_pages(s["lens"], s["more"], s["table"], s["free"], s["n_free"], page, s["slots"], s["starts"], s["status"])
        wb.kv_append(s["k"], s["v"], s["kc"], s["vc"], s["slots"])
        wb.kv_attend(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["o"])
        wb.norm_quant(s["o"].view(R, -1), None, s["codes"], s["scales"], group=128)

    a, b = fresh(), fresh()
    step(b)                                                  # (more is 0: nothing changes)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(b)
    torch.cuda.synchronize()
    g = torch.Generator().manual_seed(22)
    for more in ([60, 0, 33, 5], [1, 64, 1, 1], [1, 1, 1, 1], [64, 64, 64, 64], [1, 0, 0, 1], [64, 2, 64, 64], [1, 1, 1, 1]):
        new = dict(more=torch.tensor(more, dtype=torch.int32), k=rand(g, 64 * R, H, D).bfloat16(), v=rand(g, 64 * R, H, D).bfloat16(),
                   q=rand(g, R, H * G, D).bfloat16())
        for s in (a, b):
            for n, x in new.items():
                s[n].copy_(x)
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        assert int(a["status"]) == 0 and a["lens"].cpu().tolist() == b["lens"].cpu().tolist()
        for n in ("kc", "vc", "table", "n_free", "slots", "starts", "status", "o", "codes", "scales"):
            x, y = (s[n].view(torch.uint8) if s[n].element_size() == 1 else s[n] for s in (a, b))
            assert torch.equal(x, y), (n, more)
        float(a["o"].float().sum())                          # eager work between the replays


def test_calls_on_two_streams_do_not_disturb_each_other():
    """The same call on two streams at once, each with a workspace of its own, and on a stream
    that is passed instead of made current."""
    import linear_attn_decode_amd as wb
    g = torch.Generator().manual_seed(5)
    page, H, D, width, R = 64, 2, 128, 80, 2
    runs = []
    for i in range(2):
        k, _ = random_cache(g, R * width, H, page, D, "bf16")
        v, _ = random_cache(g, R * width, H, page, D, "bf16")
        q = rand(g, R, 8 * H, D, dtype="bf16").cuda()
        table = torch.randperm(R * width, generator=g).int().view(R, width).cuda()
        lens = torch.tensor([5000 - 700 * i, 4321], dtype=torch.int32).cuda()
        want = torch.empty_like(q)
        wb.kv_attend(q, k, v, table, lens, want)
        runs.append((q, k, v, table, lens, torch.empty_like(q), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for q, k, v, table, lens, o, want, s in runs:
            o.zero_()
        torch.cuda.synchronize()
        for n, (q, k, v, table, lens, o, want, s) in enumerate(runs):
            if n:
                wb.kv_attend(q, k, v, table, lens, o, stream=s)
            else:
                with torch.cuda.stream(s):
                    wb.kv_attend(q, k, v, table, lens, o)
        torch.cuda.synchronize()
        for q, k, v, table, lens, o, want, s in runs:
            assert torch.equal(o, want)


def test_two_captured_calls_replay_side_by_side():
    """Two graphs of the same call on other inputs, replayed on two streams at once: each has a
    workspace of its own, and every replay the eager call's bits."""
    import linear_attn_decode_amd as wb
    g = torch.Generator().manual_seed(31)
    page, H, D, width, R = 16, 8, 128, 64, 6
    k, v = (rand(g, R * width, H, page, D, dtype="bf16").cuda() for _ in range(2))
    table = torch.randperm(R * width, generator=g).int().view(R, width).cuda()
    runs = []
    for i in range(2):
        q = rand(g, R, 4 * H, D, dtype="bf16").cuda()
        lens = torch.tensor([1000 - 300 * i, 5, 700, 1024, 0, 333 + i], dtype=torch.int32).cuda()
        want, o = torch.empty_like(q), torch.zeros_like(q)
        wb.kv_attend(q, k, v, table, lens, want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                wb.kv_attend(q, k, v, table, lens, o)
        runs.append((graph, o, want, torch.cuda.Stream(), q, lens))
    for _ in range(10):
        for _, o, *_ in runs:
            o.zero_()
        torch.cuda.synchronize()
        for graph, o, want, s, *_ in runs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for graph, o, want, *_ in runs:
            assert torch.equal(o, want)
        wb.kv_attend(runs[0][4], k, v, table, runs[0][5], torch.empty_like(runs[0][1]))      # eager work between


@pytest.mark.parametrize("D,H", [(128, 4), (64, 2), (256, 4)])
def test_attend_workspace_may_hold_anything(D, H):
    """The same call with workspaces of zeros, ones, noise and what earlier calls (also of other
    sizes) left there: equal results."""
    import linear_attn_decode_amd as wb
    from linear_attn_decode_amd import serve as S
    g = torch.Generator().manual_seed(9)
    page, width, R = 16, 60, 7
    k, v = (rand(g, R * width, H, page, D, dtype="bf16").cuda() for _ in range(2))
    table = torch.randperm(R * width, generator=g).int().view(R, width).cuda()
    q = rand(g, R, 4 * H, D, dtype="bf16").cuda()
    all_lens = [[960, 5, 0, 700, 31, 128, 400], [1, 2, 3, 4, 5, 6, 7], [960] * 7]
    want = []
    for lens in all_lens:
        o = torch.empty_like(q)
        wb.kv_attend(q, k, v, table, torch.tensor(lens, dtype=torch.int32).cuda(), o)
        want.append(o)
    torch.cuda.synchronize()
    c, dev, shape, code = S._cache(k, v, None, None)
    n = S._attend_work(code, *shape, R, 4 * H, width)
    assert n > 0
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    for fill in (0, 255, None, "left", "left"):
        if fill is None:
            work.copy_(torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8))
        elif fill != "left":
            work.fill_(fill)
        for lens, o_want in zip(all_lens, want):
            o = torch.zeros_like(q)
            ln = torch.tensor(lens, dtype=torch.int32).cuda()
            S._call("kv_attend", dev, c, q.data_ptr(), 4 * H * D, D, code, R, 4 * H, table.data_ptr(), width, ln.data_ptr(),
                    D ** -0.5, 0, o.data_ptr(), None, work.data_ptr(), n, S._stream_of(dev, None))
            torch.cuda.synchronize()
            assert torch.equal(o, o_want), (fill, lens)


def test_binding_refusals():
    import linear_attn_decode_amd as wb
    cu = lambda *a, **kw: torch.zeros(*a, device="cuda", **kw)
    bf, f8, i32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32
    k, q, t, n = cu((4, 2, 16, 64), dtype=bf), cu((3, 4, 64), dtype=bf), cu((3, 2), dtype=i32), cu(3, dtype=i32)
    o = torch.empty_like(q)
    with pytest.raises(ValueError, match="v_cache"):
        wb.kv_attend(q, k, k[:3], t, n, o)
    with pytest.raises(ValueError, match="only a float8_e4m3fn cache"):
        wb.kv_attend(q, k, k, t, n, o, k_scale=cu((4, 2, 16)), v_scale=cu((4, 2, 16)))
    with pytest.raises(ValueError, match="needs the scales"):
        wb.kv_attend(q, k.to(f8), k.to(f8), t, n, o)
    with pytest.raises(ValueError, match="lens"):
        wb.kv_attend(q, k, k, t, n.long(), o)
    with pytest.raises(ValueError, match="table"):
        wb.kv_attend(q, k, k, t[:2], n, o)
    with pytest.raises(ValueError, match="o: expected"):
        wb.kv_attend(q, k, k, t, n, o.half())
    with pytest.raises(ValueError, match="contiguous heads"):
        wb.kv_attend(q.transpose(1, 2), k, k, t, n, o)
    with pytest.raises(ValueError, match="q, table"):
        wb.kv_attend(q[0], k, k, t, n, o)
    with pytest.raises(RuntimeError, match="EUNSUPPORTED"):
        wb.kv_attend(q.half(), k, k, t, n, o.half())
    with pytest.raises(RuntimeError, match="EINVAL"):
        wb.kv_attend(q[:, :3], k, k, t, n, o[:, :3].contiguous())
    with pytest.raises(RuntimeError, match="EALIGN"):
        wb.kv_attend(cu((3, 4, 65), dtype=bf)[:, :, 1:], k, k, t, n, o)
    with pytest.raises(ValueError, match="k: expected"):
        wb.kv_append(q, q, k, k, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="slots"):
        wb.kv_append(q[:, :2].contiguous(), q[:, :2].contiguous(), k, k, n)
    with pytest.raises(ValueError, match="codes"):
        wb.norm_quant(cu((2, 8)), None, cu((2, 8)), cu((2, 1)))
    with pytest.raises(ValueError, match="there is no residual"):
        wb.norm_quant(cu((2, 8)), None, cu((2, 8)).to(f8), cu((2, 1)), residual_out=cu((2, 8)))
    with pytest.raises(ValueError, match="weight"):
        wb.norm_quant(cu((2, 8)), cu(8, dtype=bf), cu((2, 8)).to(f8), cu((2, 1)))
    with pytest.raises(RuntimeError, match="EUNSUPPORTED"):
        wb.norm_quant(cu((2, 8)), None, cu((2, 8)).to(f8), cu((2, 2)), group=4)
    with pytest.raises(ValueError, match="slots"):
        wb.plan_pages(n, n, t, cu(8, dtype=i32), cu(1, dtype=i32), 16, cu(3, dtype=i32), cu(4, dtype=i32), cu(1, dtype=i32))
