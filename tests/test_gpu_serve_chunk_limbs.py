"""kv_attend_chunk with weights as two 16-bit limbs and as one (include/wbserve.h: WB_ONE_LIMB; the binding's limbs).

Bounds as in tests/test_gpu_serve_chunk.py, with the rounding r of a weight by its two limbs: 2^-16 in bfloat16 (half a step
of half a step, 2^-8 each), 2^-21 in float16 (2^-22, and 2^-36 of the largest weight where the second limb is below the
normal numbers); by one: 2^-8 and 2^-11."""
import math

import numpy as np
import pytest

from oracle import serving as O
from tests.test_gpu_serve_chunk import NEWS, PASTS, TYPES, U, make_table, rand, random_cache, stored64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
KINDS = [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")]


def i32(a):
    return torch.tensor(np.asarray(a, np.int32)).cuda()


def problem(kv, qt, D, H, G, news, pasts, page, seed):
    g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    lens = [a + b for a, b in zip(news, pasts)]
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    pages = sum(-(-n // page) for n in lens) + 2
    table = make_table(rng, lens, page, pages, max(-(-n // page) for n in lens) + 1)
    k, ks = random_cache(g, pages, H, page, D, kv)
    v, vs = random_cache(g, pages, H, page, D, kv)
    q = rand(g, int(starts[-1]), H * G, D, dtype=qt).cuda()
    return q, k, ks, v, vs, table, lens, starts


def run(kv, qt, D, H, G, news, pasts, page, window=0, seed=0, limbs=2):
    import linear_attn_decode_amd as wb
    print(f"[case] limbs={limbs} kv={kv} q={qt} D={D} H={H} G={G} new={news[:8]} past={pasts[:8]} page={page} window={window}", flush=True)
    q, k, ks, v, vs, table, lens, starts = problem(kv, qt, D, H, G, news, pasts, page, seed)
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    wb.kv_attend_chunk(q, k, v, i32(table), i32(lens), i32(starts), o, window=window, lse=lse, k_scale=ks, v_scale=vs, limbs=limbs)
    torch.cuda.synchronize()
    k64, v64, q64 = stored64(k, ks), stored64(v, vs), q.double().cpu().numpy()
    got, got_l = o.double().cpu().numpy(), lse.double().cpu().numpy()
    half = torch.finfo(TYPES[qt]).eps / 2
    for r, n in enumerate(lens):
        rows = slice(starts[r], starts[r + 1])
        if starts[r] == starts[r + 1]:
            continue
        t = np.arange(n)
        at = table[r][t // page]
        ro, rl, W, size = O.attend_chunk(q64[rows], k64[at, :, t % page], v64[at, :, t % page], 1 / math.sqrt(D), window)
        A = max(1.0, size.max())
        e_s, sums = (D + 8) * U * A + 2.0 ** -22 * A, (96 + n / 16) * U
        weight = 2.0 ** -21 if kv == "f16" else 2.0 ** -16
        if limbs == 1 and (kv, qt) != ("e4m3", "f16"):
            weight = 2.0 ** -11 if kv == "f16" else 2.0 ** -8
        tol = half * np.abs(ro) + W * (2 * e_s + weight + 2 * sums) * (1 + half) + (2.0 ** -25 if qt == "f16" else 2.0 ** -40)
        if kv == "f16":
            tol += n * 2.0 ** -36 * np.abs(v64).max()
        assert (np.abs(got[rows] - ro) <= tol).all(), (r, n, float((np.abs(got[rows] - ro) / tol).max()))
        assert (np.abs(got_l[rows] - rl) <= e_s + sums + 2 * U * np.abs(rl)).all(), (r, n)
    again = torch.full_like(q, 7.0)
    wb.kv_attend_chunk(q, k, v, i32(table), i32(lens), i32(starts), again, window=window, k_scale=ks, v_scale=vs, limbs=limbs)
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), o.view(torch.int16))
    return o


@pytest.mark.parametrize("kv,qt", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("limbs", [2, 1])
def test_types_and_widths(kv, qt, D, limbs):
    run(kv, qt, D, 2, 4, NEWS, PASTS, 16, seed=D, limbs=limbs)
    run(kv, qt, D, 1, 5, [100, 1, 300], [700, 3, 0], 32, window=77, seed=D + 1, limbs=limbs)


@pytest.mark.parametrize("kv,qt", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("limbs", [2, 1])
def test_long_caches_are_split_and_joined(kv, qt, D, limbs):
    run(kv, qt, D, 1, 4, [7, 1], [9000, 4000], 64, seed=3, limbs=limbs)


@pytest.mark.parametrize("kv,qt", KINDS)
def test_two_limbs_unless_one_is_asked_for(kv, qt):
    import linear_attn_decode_amd as wb
    q, k, ks, v, vs, table, lens, starts = problem(kv, qt, 64, 1, 2, [40], [300], 16, 1)
    outs = [torch.empty_like(q) for _ in range(3)]
    for o, kw in zip(outs, ({}, dict(limbs=2), dict(limbs=1))):
        wb.kv_attend_chunk(q, k, v, i32(table), i32(lens), i32(starts), o, k_scale=ks, v_scale=vs, **kw)
    torch.cuda.synchronize()
    same = [torch.equal(outs[0].view(torch.int16), o.view(torch.int16)) for o in outs]
    assert same[1] and same[2] == ((kv, qt) == ("e4m3", "f16"))


def test_many_requests():
    rng = np.random.default_rng(5)
    run("bf16", "bf16", 64, 2, 2, [int(n) for n in rng.integers(0, 6, 200)], [int(n) for n in rng.integers(1, 300, 200)], 16, seed=6)


@pytest.mark.parametrize("kv,qt", KINDS)
def test_one_weight_many_times(kv, qt):
    """31 tokens of one weight, e^-1.75, beside one of value 0: o = 31 w / (1 + 31 w) within half a step and the limbs' rounding
    (2^-16; 40 u for the weight and the sums)."""
    import linear_attn_decode_amd as wb
    D, page, n = 64, 16, 32
    q = torch.zeros((1, 1, D), dtype=TYPES[qt], device="cuda")
    q[..., 0] = 1
    k = torch.zeros((2, 1, page, D), device="cuda")
    k[0, 0, 0, 0] = 1.75                                       # the others' weight is e^-1.75: between numbers of 16 bits
    v = torch.ones((2, 1, page, D), device="cuda")
    v[0, 0, 0] = 0
    k, v = k.to(TYPES[kv]), v.to(TYPES[kv])
    one = torch.ones((2, 1, page), device="cuda") if kv == "e4m3" else None
    w = math.exp(-1.75)
    want = (n - 1) * w / (1 + (n - 1) * w)
    off = {}
    for limbs in (1, 2):
        o = torch.empty_like(q)
        wb.kv_attend_chunk(q, k, v, i32([[0, 1]]), i32([n]), i32([0, 1]), o, scale=1.0, k_scale=one, v_scale=one, limbs=limbs)
        torch.cuda.synchronize()
        off[limbs] = abs(o[0, 0, 0].double().item() - want) / want
    half = torch.finfo(TYPES[qt]).eps / 2
    assert off[2] <= half * (1 + 2.0 ** -7) + 2.0 ** -16 + 40 * U, off
    assert off[1] <= half + {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -8}[kv] * (1 + half) + 40 * U, off
    if kv == "e4m3" and qt == "f16":
        assert off[1] == off[2]


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
def test_two_limbs_are_as_close_as_kv_attend(kv):
    """Single tokens: outputs of the two operators are within their roundings of one another, two half steps and the limbs' 2^-15
    of the values (at most 4 or so, 448 codes times 0.015 of an 8-bit cache: 7). They differ where a border between two outputs is
    within the limbs' error, which is 2^-8 steps of bfloat16, 2^-10 of float16: in few."""
    import linear_attn_decode_amd as wb
    qt, D, H, G, R = "bf16" if kv == "e4m3" else kv, 128, 2, 4, 40
    rng = np.random.default_rng(2)
    news, pasts = [1] * R, [int(n) for n in rng.integers(50, 3000, R)]
    o = run(kv, qt, D, H, G, news, pasts, 16, seed=9)
    q, k, ks, v, vs, table, lens, starts = problem(kv, qt, D, H, G, news, pasts, 16, 9)
    one = torch.empty_like(q)
    wb.kv_attend(q, k, v, i32(table), i32(lens), one, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    half = torch.finfo(TYPES[qt]).eps / 2
    assert ((o.double() - one.double()).abs() <= 2 * half * one.double().abs() + 2.0 ** -15 * 7).all()
    assert (o.view(torch.int16) == one.view(torch.int16)).float().mean().item() > 0.9


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("limbs", [2, 1])
def test_hidden_infinities_leave_no_trace(kv, D, limbs):
    import linear_attn_decode_amd as wb
    qt, page, H = "bf16" if kv == "e4m3" else kv, 16, 2
    q, k, ks, v, vs, table, lens, starts = problem(kv, qt, D, H, 4, [13, 45], [3, 70], page, 4)
    args = (i32(table), i32(lens), i32(starts))
    outs = []
    for spoil in (False, True):
        if spoil:
            for r, n in enumerate(lens):                     # behind each request's last token
                if n % page:
                    v[table[r][n // page], :, n % page:] = torch.full((D,), math.nan).to(v.dtype).cuda()
            later = table[1][100 // page], slice(None), 100 % page     # a token that only later rows of the second request see
            v[later] = torch.full((D,), math.nan).to(v.dtype).cuda()
        o = torch.empty_like(q)
        wb.kv_attend_chunk(q, k, v, *args, o, k_scale=ks, v_scale=vs, limbs=limbs)
        torch.cuda.synchronize()
        outs.append(o)
    sees = 13 + 100 - 70                                      # its row
    assert torch.equal(outs[0][:sees].view(torch.int16), outs[1][:sees].view(torch.int16))
    assert torch.isnan(outs[1][sees:]).all()


def test_limbs_are_one_or_two():
    import linear_attn_decode_amd as wb
    q, k, ks, v, vs, table, lens, starts = problem("bf16", "bf16", 64, 1, 1, [3], [0], 16, 0)
    for limbs in (0, 3, -1, None):
        with pytest.raises(ValueError):
            wb.kv_attend_chunk(q, k, v, i32(table), i32(lens), i32(starts), torch.empty_like(q), limbs=limbs)
