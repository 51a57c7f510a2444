"""The sum of weights of kv_attend_chunk (include/wbserve.h) over long caches that are not split: enough blocks of rows to
fill the card, flat scores below an early maximum, so that every addition of a running sum would round the same way.

u = 2^-24. Scores are exact (one product of small numbers), so an exponent gap * log2(e) is within 3 u gap log2(e), the
exponential adds 2^-22: E = 2^-22 + 4 u gap for the logarithm. A tile's weights are added in pairs and eight steps (10 u), the
tiles' sums with their remainders (2 u), the two lanes of a row and the remainder in two more additions; log adds 2 u of
itself: |lse - lse*| <= E + 16 u + 2 u |lse*|. The output is v times the weights' mean rounding: within the type's r
(2^-8 bfloat16, 2^-11 float16) and half a step of its own, and (n/16 + 16) u of the products' sums."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


@pytest.mark.parametrize("kv,qt,D", [("bf16", "bf16", 64), ("f16", "f16", 128), ("e4m3", "f16", 64), ("bf16", "bf16", 256)])
@pytest.mark.parametrize("n", [8192, 32768, 131072])
@pytest.mark.parametrize("gap", [1.5, 2.375, 0.25])
def test_flat_scores_below_an_early_maximum(kv, qt, D, n, gap):
    import linear_attn_decode_amd as wb
    print(f"[case] flat kv={kv} q={qt} D={D} n={n} gap={gap}", flush=True)
    H, G, m, page = 4, 128, 132, 64                          # 528 blocks of one token each
    pages = n // page
    q = torch.zeros((m, H * G, D), dtype=TYPES[qt], device="cuda")
    q[..., 0] = 1
    k = torch.zeros((pages, H, page, D), dtype=torch.bfloat16, device="cuda")
    k[0, :, 0, 0] = gap
    k, v = k.to(TYPES[kv]), torch.ones((pages, H, page, D), dtype=torch.bfloat16, device="cuda").to(TYPES[kv])
    gap = k[0, 0, 0, 0].float().item()                       # (as it is stored: 2.375 is no e4m3 number)
    one = torch.ones((pages, H, page), device="cuda") if kv == "e4m3" else None
    o = torch.full((m, H * G, D), 7.0, dtype=TYPES[qt], device="cuda")
    lse = torch.full((m, H * G), 7.0, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    wb.kv_attend_chunk(q, k, v, i32([list(range(pages))]), i32([n]), i32([0, m]), o, scale=1.0, lse=lse, k_scale=one, v_scale=one)
    torch.cuda.synchronize()
    seen = np.arange(n - m + 1, n + 1)
    want = gap + np.log1p((seen - 1) * math.exp(-gap))
    tol = 2.0 ** -22 + 4 * U * gap + 16 * U + 2 * U * want
    err = np.abs(lse.double().cpu().numpy() - want[:, None])
    print(f"[worst] {(err / tol[:, None]).max():.3f} of the bound", flush=True)
    assert (err <= tol[:, None]).all(), err.max()
    r = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -16}[kv]
    assert ((o.double() - 1).abs() <= torch.finfo(TYPES[qt]).eps / 2 + r + 2 * (n / 16 + 16) * U).all()


@pytest.mark.parametrize("kv,qt", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16")])
def test_sums_follow_a_rising_maximum(kv, qt):
    """Maxima that rise by 5 a tile or so: the remainders move with the sums. (Each move multiplies both by one rounded
    factor: 2^-22 and u for each of the 1024 moves' products, of sums of which the moves leave e^-5: 1.01 of one.)"""
    import linear_attn_decode_amd as wb
    H, G, m, page, D, n = 4, 128, 132, 64, 64, 16384
    pages = n // page
    q = torch.zeros((m, H * G, D), dtype=TYPES[qt], device="cuda")
    q[..., 0] = 1
    step = torch.arange(n) // 512 * 5.0                      # (0 .. 155: exact in each type but by quarters of 448 codes)
    if kv == "e4m3":
        step = torch.arange(n) // 2048 * 8.0                 # (0 .. 56)
    k = torch.zeros((pages, page, H, D))
    k[..., 0] = step.view(pages, page, 1)
    k = k.transpose(1, 2).contiguous().cuda().to(TYPES[kv])
    assert torch.equal(k[:, 0, :, 0].float().cpu().flatten(), step)
    v = torch.ones_like(k, dtype=torch.bfloat16).to(TYPES[kv])
    one = torch.ones((pages, H, page), device="cuda") if kv == "e4m3" else None
    o, lse = torch.empty_like(q), torch.empty((m, H * G), device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    wb.kv_attend_chunk(q, k, v, i32([list(range(pages))]), i32([n]), i32([0, m]), o, scale=1.0, lse=lse, k_scale=one, v_scale=one)
    torch.cuda.synchronize()
    x = step.double().numpy()
    want = np.array([x[:s].max() + math.log(np.exp(x[:s] - x[:s].max()).sum()) for s in range(n - m + 1, n + 1)])
    tol = 2.0 ** -16 + 2 * 2.0 ** -22 + 20 * U + 2 * U * want
    assert (np.abs(lse.double().cpu().numpy() - want[:, None]) <= tol[:, None]).all()
