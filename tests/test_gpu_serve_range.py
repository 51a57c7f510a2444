"""The serving operators (include/wbserve.h) where their numbers and sizes come near the ends
of their ranges, against their float64 definitions (oracle/serving.py).

Tolerances, from the arithmetic (u = 2^-24, half a float32 step), are written at each test.
"""
import math

import numpy as np
import pytest

from oracle import serving as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------- attention
def sink_bound(ro, W, n, D, gap, kv, v_max):
    """Scores are within e_s = (D + 4) u A + 2^-22 A (A: the largest, `gap`), a weight and the
    sum that divides it off by that each, sums over tokens by (96 + n / 32) u twice; a weight's
    limbs leave 2^-17 of it, float16 ones also half of the smallest float16 step at 2^15 times
    the weight, 2^-40 a token; the output is rounded once, by half a step, which is not below
    2^-25 in float16."""
    A = max(1.0, abs(gap))
    e_s = (D + 4) * U * A + 2.0 ** -22 * A
    half = torch.finfo(TYPES[kv]).eps / 2 * np.abs(ro)
    tol = W * (2 * e_s + 2.0 ** -17 + 2 * (96 + n / 32) * U)
    if kv == "f16":
        half, tol = np.maximum(half, 2.0 ** -25), tol + n * 2.0 ** -40 * v_max
    return half + tol


@pytest.mark.parametrize("gap", [9.0, 12.0, 15.0, 16.5, 17.0, 17.5, 18.0])
@pytest.mark.parametrize("kv,D,R,n,at", [("f16", 256, 800, 2048, 0), ("f16", 64, 1, 20000, 0), ("f16", 128, 1, 20000, 9000),
                                         ("f16", 128, 3, 131072, 1), ("bf16", 128, 1, 20000, 0)])
def test_attend_one_token_far_above_all_others(kv, D, R, n, at, gap):
    """A token of value 0 that takes nearly all the weight, `gap` above n - 1 equal ones that
    make up the row: whole requests of one workgroup (800 of 16 turns on 256 workgroups) and
    split ones. The requests share their pages."""
    import linear_attn_decode_amd as wb
    print(f"[case] sink kv={kv} D={D} R={R} n={n} at={at} gap={gap}", flush=True)
    page = 64
    pages = -(-n // page)
    k = torch.zeros((pages, 1, page, D), dtype=TYPES[kv], device="cuda")
    v = torch.full_like(k, 64.0)
    k[at // page, 0, at % page, 0] = gap
    v[at // page, 0, at % page] = 0
    q = torch.zeros((R, 2, D), dtype=TYPES[kv], device="cuda")
    q[:, 0, 0], q[:, 1, 0] = 1.0, 0.5                                    # (the second head: half the gap)
    table = torch.arange(pages, dtype=torch.int32).repeat(R, 1).cuda()
    o, lse = torch.empty_like(q), torch.empty((R, 2), device="cuda")
    wb.kv_attend(q, k, v, table, torch.full((R,), n, dtype=torch.int32).cuda(), o, scale=1.0, lse=lse)
    torch.cuda.synchronize()
    for h, g in ((0, gap), (1, gap / 2)):
        rest = (n - 1) * math.exp(-g)
        ro = 64.0 * rest / (1 + rest)
        got = o[:, h].double().cpu().numpy()
        assert (np.abs(got - ro) <= sink_bound(ro, ro, n, D, g, kv, 64.0)).all(), (h, ro, got.min(), got.max())
        want = g + math.log1p(rest)
        e_s = (D + 4) * U * g + 2.0 ** -22 * g
        assert (np.abs(lse[:, h].double().cpu().numpy() - want) <= e_s + (96 + n / 32) * U + 2 * U * want).all()


@pytest.mark.parametrize("n", [1, 300, 5000])
def test_attend_largest_float16_values(n):
    """Equal weights over the largest values: the sums of 2^15 times the weights stay float32
    numbers, and the mean is the value (off by (96 + n / 32) u, far below half a float16 step)."""
    import linear_attn_decode_amd as wb
    page, D = 64, 128
    pages = -(-n // page)
    k = torch.zeros((pages, 1, page, D), dtype=torch.float16, device="cuda")
    v = torch.full_like(k, 65504.0)
    v[..., 1::2] = -65504.0
    q = torch.ones((1, 4, D), dtype=torch.float16, device="cuda")
    o = torch.empty_like(q)
    wb.kv_attend(q, k, v, torch.arange(pages, dtype=torch.int32)[None].cuda(), torch.tensor([n], dtype=torch.int32).cuda(), o)
    torch.cuda.synchronize()
    assert (o[..., ::2] == 65504).all() and (o[..., 1::2] == -65504).all()


def test_attend_weights_of_random_scores_far_apart():
    """Float16 keys whose scores spread over some 30 nats, against the definition, without an
    allowance for lost weights but 2^-40 a token."""
    import linear_attn_decode_amd as wb
    page, D, H, G, n = 16, 64, 2, 4, 6000
    g = torch.Generator().manual_seed(41)
    pages = n // page
    k, v = (torch.randn((pages, H, page, D), generator=g).half().cuda() for _ in range(2))
    q = (4 * torch.randn((1, H * G, D), generator=g)).half().cuda()
    o = torch.empty_like(q)
    wb.kv_attend(q, k, v, torch.arange(pages, dtype=torch.int32)[None].cuda(), torch.tensor([n], dtype=torch.int32).cuda(), o)
    torch.cuda.synchronize()
    k64, v64 = (x.double().cpu().numpy().transpose(0, 2, 1, 3).reshape(n, H, D) for x in (k, v))
    ro, _, W, size = O.attend(q[0].double().cpu().numpy(), k64, v64, D ** -0.5)
    err = np.abs(o[0].double().cpu().numpy() - ro)
    tol = sink_bound(ro, W, n, D, float(size.max()), "f16", np.abs(v64).max())
    assert (err <= tol).all(), float((err / tol).max())


# ---------------------------------------------------------------------------- norm
# every kernel: 8, 16, 32 and 64 lanes a row, a workgroup with 2, 4 and 8 chunks a lane
NORM_WIDTHS = [1, 50, 100, 200, 500, 1000, 5000, 20000, 40000]


@pytest.mark.parametrize("D", NORM_WIDTHS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_rows_of_zeros_without_eps(D, dt):
    """A group of zeros has scale 0 and codes 0, with eps = 0 too, beside rows that are not zero."""
    import linear_attn_decode_amd as wb
    print(f"[case] norm zeros D={D} {dt}", flush=True)
    x = torch.ones((5, D), dtype=TYPES[dt], device="cuda")
    x[0] = x[3] = 0
    w = torch.full((D,), -2.0, dtype=TYPES[dt], device="cuda")
    r = torch.zeros_like(x)
    for group in (0, 128):
        codes = torch.empty((5, D), dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty((5, -(-D // group) if group else 1), device="cuda")
        for kw in ({}, {"residual": r, "residual_out": torch.empty_like(x)}):
            codes.view(torch.uint8).fill_(77)
            scales.fill_(math.nan)
            wb.norm_quant(x, w, codes, scales, eps=0.0, group=group, **kw)
            torch.cuda.synchronize()
            c = codes.float()
            assert (c[[0, 3]] == 0).all() and (scales[[0, 3]] == 0).all()
            assert (c[[1, 2, 4]] == -448).all() and (scales[[1, 2, 4]] - 2 / 448).abs().max() <= 2 / 448 * 8 * U


def check_norm(x, w, eps, group, residual=None):
    """A row's squares are all positive: their sum is off by a step a value of a lane (64 at
    most), a step of lanes (6) and a wavefront (16), and y takes half of that and 24 more
    roundings; y and products below the normal numbers are off by 2^-150 each, 2^-23 of the least
    scale, three of them; a code by half a step, in doubt by those."""
    import linear_attn_decode_amd as wb
    N, D = x.shape
    assert w is None or float(w.abs().max()) <= 1.9
    codes = torch.empty((N, D), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((N, -(-D // group) if group else 1), device="cuda")
    out = None if residual is None else torch.empty_like(x)
    wb.norm_quant(x, w, codes, scales, eps=eps, group=group, residual=residual, residual_out=out)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        h, y, want = O.norm(x.double().cpu().numpy(), None if residual is None else residual.double().cpu().numpy(),
                            None if w is None else w.double().cpu().numpy(), float(np.float32(eps)), group)
    zeros = (h == 0).all(1)                                              # (0 / 0 without eps: by the interface, 0)
    y[zeros], want[zeros] = 0, 0
    if residual is not None:
        t = torch.finfo(x.dtype).eps
        assert (np.abs(out.double().cpu().numpy() - h) <= (t / 2 + 2 * U) * np.abs(h)).all()
    rel = (86 + 24) * U
    sc = scales.double().cpu().numpy()
    # (1 / rms is 2^k in [1, 2) times: h 2^k of 2^-150 and less is 0 in float32, with weights up to
    # 1.9 here a y of up to 2^-148.07, and a group of such values one of zeros)
    top = np.stack([np.abs(y[:, i:i + (group or D)]).max(1) for i in range(0, D, group or D)], 1)
    nothing = (sc == 0) & (top <= 2.0 ** -148)
    assert (nothing | (np.abs(sc - want) <= (rel + 2 * U) * want)).all(), (sc[:, 0], want[:, 0])
    q = np.clip(y / np.repeat(np.where(sc > 0, sc, 1.0), group or D, axis=1)[:, :D], -448, 448)
    err = np.abs(codes.double().cpu().numpy() - q)
    assert (err <= O.e4m3_half_step(q) + 2 * rel * np.abs(q) + 3 * 2.0 ** -23).all()


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-30, 1e-6, 1e30])
@pytest.mark.parametrize("D", NORM_WIDTHS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_rows_whose_squares_leave_the_range(dt, D, eps):
    """Rows near the largest and the smallest numbers, whose squares are infinite or 0 in
    float32, each beside an ordinary one, and rows that hold both ends."""
    print(f"[case] norm range {dt} D={D} eps={eps}", flush=True)
    g = torch.Generator().manual_seed(D)
    size = [1.0, 2.0 ** 124, 2.0 ** 64, 2.0 ** 63, 1.0, 2.0 ** -48, 2.0 ** -60, 2.0 ** -64, 2.0 ** -75, 2.0 ** -110, 2.0 ** -126,
            2.0 ** -146 if dt == "f32" else 2.0 ** -130, 1.0]
    x = (torch.randn((len(size), D), generator=g).clamp(-4, 4).double() * torch.tensor(size, dtype=torch.float64)[:, None]).to(TYPES[dt])
    x[4, ::3] = 2.0 ** 100
    x[12, ::3] = 2.0 ** -80
    w = (1 + 0.3 * torch.rand(D, generator=g)).to(TYPES[dt])
    check_norm(x.cuda(), w.cuda(), eps, 128)
    check_norm(x.cuda(), None, eps, 0)
    check_norm(x.cuda(), w.cuda(), eps, 0, residual=torch.zeros_like(x).cuda())


def test_norm_weight_that_is_the_rows_is_refused():
    """A weight is [D], also where the rows themselves are given for one."""
    import linear_attn_decode_amd as wb
    wide = torch.ones((2, 16), device="cuda")
    for x in (wide, wide[:, :8], wide[:1]):
        codes, scales = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((x.shape[0], 1), device="cuda")
        with pytest.raises(ValueError, match="weight"):
            wb.norm_quant(x, x, codes, scales)


# ---------------------------------------------------------------------------- sizes
@pytest.fixture
def large():
    """Memory for tests of many rows, given back behind them."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 130 GB of free GPU memory")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N,D", [(2 ** 29 + 5, 1), (2 ** 28 + 1, 65), (2 ** 26 + 3, 513)])
def test_norm_of_more_rows_than_a_grid_dimension_holds(large, N, D):
    """8, 16 and 64 lanes a row, 2^32 of them and more: rows of zeros, but for some."""
    import linear_attn_decode_amd as wb
    print(f"[case] norm N={N} D={D}", flush=True)
    x = torch.zeros((N, D), dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 2 ** 25 - 1, 2 ** 25, N // 2, N - 2, N - 1]
    for i, r in enumerate(at):
        x[r] = i + 1
    codes = torch.empty((N, D), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.full((N, 1), math.nan, device="cuda")
    wb.norm_quant(x, None, codes, scales, eps=0.0)
    torch.cuda.synchronize()
    assert int((scales == 0).sum()) == N - len(at)
    for r in at:
        # (y is 1 but for the roundings of the sum, the root and the products: 110 u, as above)
        assert abs(float(scales[r]) * 448 - 1) <= 112 * U and (codes[r].float() == 448).all()
    for r in {2, 3, 2 ** 25 + 1, N - 3} - set(at):
        assert (codes[r].float() == 0).all()


def test_append_of_more_vectors_than_a_grid_dimension_holds(large):
    """2^27 vectors of 32 lanes and more, all but some of them padding. (Keys and values are the
    same memory here: they are only read.)"""
    import linear_attn_decode_amd as wb
    N, H, D, page = 2 ** 21 + 9, 64, 256, 8
    print(f"[case] append N={N} H={H} D={D}", flush=True)
    k = torch.empty((N, H, D), dtype=torch.bfloat16, device="cuda")
    slots = torch.full((N,), -1, dtype=torch.int64, device="cuda")
    at = [0, 5, 2 ** 20, 2 ** 21 - 1, 2 ** 21, N - 1]
    g = torch.Generator().manual_seed(51)
    new = torch.randn((len(at), H, D), generator=g).bfloat16().cuda()
    for i, r in enumerate(at):
        k[r] = new[i]
        slots[r] = 2 * i + 1
    kc, vc = (torch.full((2, H, page, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wb.kv_append(k, k, kc, vc, slots)
    torch.cuda.synchronize()
    want = torch.full((2 * page, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    want[torch.arange(len(at)).cuda() * 2 + 1] = new
    want = want.view(2, page, H, D).transpose(1, 2)
    assert torch.equal(kc, want) and torch.equal(vc, want)
