"""GPU parity of token_logprobs (include/wbserve.h) with its float64 definition (oracle/serving.py).

Tolerance, from the arithmetic (u = 2^-24, half a float32 step). With d = scale (max - x), an exponent is
(x - m) * (scale log2 e): within 3 u of |d|, the exponential within 4 u: e = (3 d + 4) u of a weight, which
counts by its weight (E = sum p d). A lane adds V / 512 weights, then 6 + 8 + 64 sums are joined, each after a
move of the maximum (3 u): n = (V / 512 + 4 * 96) u. So
  |logprob - *| <= (3 E + 4) u + n + 3 u (d_token + |log s|),
  |entropy - *| <= (3 E + 4) u + n + 2 u |log s| + (3 E2 + 4 E) u + 2 n E + 4 u E,  E2 = sum p d^2.
The columns are equal.
"""
import math

import numpy as np
import pytest

from oracle import serving as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def run(x, tokens, K, scale=1.0, wide=True, rows=None):
    """x: logits on the GPU, perhaps strided; the oracle checks `rows` of them (all)."""
    import linear_attn_decode_amd as wb
    N, V = x.shape
    print(f"[case] logprobs {x.dtype} N={N} V={V} K={K} scale={scale} stride={x.stride(0)}", flush=True)
    t = torch.tensor(tokens, dtype=torch.int64 if wide else torch.int32).cuda()
    lp, en = (torch.full((N,), 7.0, device="cuda") for _ in range(2))
    ids = torch.full((N, K), -7, dtype=torch.int32, device="cuda") if K else None
    tops = torch.full((N, K), 7.0, device="cuda") if K else None
    wb.token_logprobs(x, t, lp, entropy=en, top_ids=ids, top_logprobs=tops, scale=scale)
    torch.cuda.synchronize()
    worst = 0.0
    for r in range(N) if rows is None else rows:
        y = x[r].double().cpu().numpy()
        want, entropy, order, p = O.logprobs(y, tokens[r], K, scale)
        if K:
            assert np.array_equal(ids[r].cpu().numpy(), order), (r, ids[r], order)
        got = lp[r].item(), en[r].item()
        if np.isnan(entropy):
            assert np.isnan(got).all() and (not K or torch.isnan(tops[r]).all()), (r, got)
            continue
        with np.errstate(all="ignore"):
            d = scale * (y.max() - y)
            w = np.exp(-d)
            log_s = math.log(w.sum())
            w /= w.sum()
            E, E2 = (float(np.where(w > 0, w * d ** i, 0).sum()) for i in (1, 2))
        n = (V / 512 + 384) * U
        base = (3 * E + 4) * U + n
        assert abs(got[1] - entropy) <= base + 2 * U * abs(log_s) + (3 * E2 + 4 * E) * U + 2 * n * E + 4 * U * E, (r, got, entropy)
        for a, b in [(got[0], want)] + ([(tops[r, i].item(), p[i]) for i in range(K)] if K else []):
            if np.isnan(b) or np.isinf(b):
                assert np.array_equal(a, b, equal_nan=True), (r, a, b)
            else:
                tol = base + 3 * U * (abs(b) + 2 * abs(log_s))
                assert abs(a - b) <= tol, (r, a, b, tol)
                worst = max(worst, abs(a - b) / tol)
    print(f"[worst] {worst:.3f} of the bound", flush=True)
    return lp, en, ids, tops


def logits(dtype, N, V, seed=0, slack=0, by=3.0):
    g = torch.Generator().manual_seed(seed)
    return (by * torch.randn((N, V + slack), generator=g)).to(TYPES[dtype]).cuda()[:, :V]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 511, 512, 513, 4095, 5000, 65537])
def test_types_and_sizes(dtype, V):
    rng = np.random.default_rng(V)
    for K, slack in ((min(V, 64), 0), (min(V, 5), 3), (0, 1)):
        tokens = [int(i) for i in rng.integers(0, V, 5)]
        run(logits(dtype, 5, V, seed=V + K, slack=slack), tokens, K, wide=K != 5)


@pytest.mark.parametrize("N,V", [(1, 128000), (3, 262144), (1, 2 ** 21 + 5), (40, 50001), (300, 30000), (1100, 20001)])
def test_rows_and_segments(N, V):
    """Rows in segments joined by the last, and rows of a workgroup each."""
    rng = np.random.default_rng(N)
    rows = sorted({0, N // 2, N - 1} | {int(i) for i in rng.integers(0, N, 8)})
    run(logits("bf16", N, V, seed=N, slack=1), [int(i) for i in rng.integers(0, V, N)], 20, rows=rows)
    run(logits("f32", N, V, seed=N + 1), [int(i) for i in rng.integers(0, V, N)], 64, rows=rows)


@pytest.mark.parametrize("N", [2, 2000])
@pytest.mark.parametrize("V", [700, 3000, 40000, 140000])
def test_orders_that_fill_every_stage(N, V):
    """Constant rows, rising and falling ones, a few values many times, all but some columns at -infinity:
    equal logits by their column, and many candidates."""
    i = torch.arange(V, dtype=torch.float32)
    kinds = [torch.zeros(V), -i / V, i / V, -(i // 700) / 8, (i % 3) * 0.5, torch.where(i % 997 == 5, i / V, torch.tensor(-math.inf)),
             torch.where(i == 77, 1.0, -math.inf), torch.where(i < 600, 0.0, -0.0), torch.where(i >= V - 9, 5.0, -5.0),
             torch.full((V,), torch.finfo(torch.float32).min).index_fill(0, torch.tensor([V - 1]), 0.0)]
    x = torch.stack([kinds[r % len(kinds)] for r in range(N)]).cuda()
    tokens = [(77, 0, V - 1, 5)[r % 4] for r in range(N)]
    for K in (64, 32, 3):
        run(x, tokens, K, rows=range(min(N, 10)))


@pytest.mark.parametrize("N", [3, 1500])
def test_padding_and_rows_without_probabilities(N):
    V = 9000
    x = logits("f32", N, V)
    x[0, 100] = math.nan
    x[1] = -math.inf
    x[2, 8999] = math.inf
    run(x, [V, 3, -1] + [-1] * (N - 3), 6, rows=range(min(N, 5)))


@pytest.mark.parametrize("scale", [0.25, 1.0, 7.0, 2.0 ** -100])
def test_scales(scale):
    run(logits("f16", 4, 5001), [0, 5000, 2500, 1], 8, scale=scale)


def test_far_logits():
    run(logits("bf16", 4, 5001, by=1e4), [0, 5000, 2500, 1], 8)
    run(logits("f32", 4, 5001, by=1e30), [0, 5000, 2500, 1], 8, scale=2.0 ** -90)


def test_no_rows_and_no_alternatives():
    import linear_attn_decode_amd as wb
    z = torch.zeros((0, 9), device="cuda")
    wb.token_logprobs(z, torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, device="cuda"))
    lp = torch.zeros(1, device="cuda")
    wb.token_logprobs(torch.zeros((1, 4), device="cuda"), torch.tensor([2]).cuda(), lp)
    assert abs(lp.item() + math.log(4)) < 1e-6


def test_equal_calls_give_equal_bits_and_replays_follow_their_inputs():
    import linear_attn_decode_amd as wb
    g = torch.Generator().manual_seed(5)
    x = (3 * torch.randn((2, 100000), generator=g)).cuda()
    t = torch.tensor([5, 99999]).cuda()
    outs = [(torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), torch.empty((2, 20), dtype=torch.int32, device="cuda"),
             torch.empty((2, 20), device="cuda")) for _ in range(2)]
    call = lambda o: wb.token_logprobs(x, t, o[0], entropy=o[1], top_ids=o[2], top_logprobs=o[3])
    call(outs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[1])
    for _ in range(6):
        x.copy_(3 * torch.randn(x.shape, generator=g))
        call(outs[0])
        for o in outs[1]:
            o.fill_(7)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.equal(a, b)
