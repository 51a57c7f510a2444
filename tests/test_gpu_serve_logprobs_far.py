"""token_logprobs (include/wbserve.h) where scale * logit is large or leaves float32's range: small temperatures, vocabularies
masked with the lowest finite value, tokens forced with the largest. Tolerances are those of the ordinary rows
(tests/test_gpu_serve_logprobs.py): a weight's exponent is a difference, within 3 u of itself, however large its terms."""
import math

import numpy as np
import pytest

from tests.test_gpu_serve_logprobs import TYPES, logits, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
SIZES = [(5, 5001), (300, 700), (2, 140000), (1, 2 ** 20 + 3)]               # rows of a workgroup each, rows in segments


def columns(V, seed, n):
    return [int(i) for i in np.random.default_rng(seed).integers(0, V, n)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [1e5, 1e6, 2.0 ** 22, 1e7, 1e8, 1e9, 1e10, 1e12, 2.0 ** 60, 2.0 ** 100])
def test_small_temperatures(dtype, scale):
    for (N, V), K in zip(SIZES, (8, 64, 20, 0)):
        x = logits(dtype, N, V, seed=N)
        tokens = columns(V, 1, N)
        tokens[0] = int(x[0].float().argmax())
        run(x, tokens, K, scale=scale, rows=range(min(N, 5)))


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exponent", [20, 24, 25, 26, 27, 30, 31, 35, 60, 100, 126])
def test_logits_around_a_large_one(sign, exponent):
    """float32 logits a few units in the last place apart, by a scale that makes those 1 / 4."""
    step = 2.0 ** (exponent - 23)
    for (N, V), K in zip(SIZES, (3, 0, 20, 8)):
        near = torch.randint(0, 64, (N, V), generator=torch.Generator().manual_seed(exponent)).float()
        x = (sign * (2.0 ** exponent + near * step)).cuda()
        if 2.0 ** -100 <= 0.25 / step <= 2.0 ** 100:
            run(x, columns(V, 2, N), K, scale=0.25 / step, rows=range(min(N, 3)))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [0.5, 1.0, 10.0, 1e3])
def test_rows_of_the_lowest_value(dtype, scale):
    """A vocabulary that is masked throughout is uniform; one that is but for a few columns is theirs."""
    for (N, V), K in zip(SIZES, (8, 0, 20, 64)):
        x = torch.full((N, V), torch.finfo(TYPES[dtype]).min, dtype=TYPES[dtype], device="cuda")
        lp, en, *_ = run(x, columns(V, 3, N), K, scale=scale, rows=range(min(N, 3)))
        assert (lp + math.log(V)).abs().max().item() < 1e-4 and (en - math.log(V)).abs().max().item() < 1e-4
        for at in (0, V // 3, V - 1):
            x[:, at] = 2.0
            x[:, (at + 600) % V] = 1.0
        t = [V // 3] * N
        _, _, ids, _ = run_overflowing(x, t, 6, scale)
        assert sorted(ids[0, :6].tolist()) == sorted({0, V // 3, V - 1, 600 % V, (V // 3 + 600) % V, 599})


def run_overflowing(x, tokens, K, scale):
    """As run() for log probabilities that may be past float32's range (-infinity then): all rows are alike."""
    import linear_attn_decode_amd as wb
    N, V = x.shape
    lp, en = (torch.full((N,), 7.0, device="cuda") for _ in range(2))
    ids, tops = torch.full((N, K), -7, dtype=torch.int32, device="cuda"), torch.full((N, K), 7.0, device="cuda")
    wb.token_logprobs(x, torch.tensor(tokens).cuda(), lp, entropy=en, top_ids=ids, top_logprobs=tops, scale=scale)
    torch.cuda.synchronize()
    y = x[0].double().cpu().numpy()
    p = scale * (y - y.max())
    p -= math.log(np.exp(p).sum())
    order = np.lexsort((np.arange(V), -y))[:K]
    # ((3 E + 4) u + (V / 512 + 384) u of the sum, E below 1, and 3 u of the distance)
    tol = lambda b: (V / 512 + 400) * 2.0 ** -24 + 4 * 2.0 ** -24 * abs(b)
    for got, want in [(lp, p[tokens[0]])] + [(tops[:, i], p[order[i]]) for i in range(K)]:
        ends = torch.finfo(torch.float32).max * (1 + 4 * 2.0 ** -24 * np.array([-1, 1]))        # (4 u off: either side)
        if abs(want) > ends[1]:
            assert (got == -math.inf).all(), (got, want)
        elif abs(want) > ends[0]:
            assert (got <= -ends[0]).all(), (got, want)
        else:
            assert (got.double() - want).abs().max().item() <= tol(want), (got, want)
    w = np.exp(p)
    entropy = -np.where(w > 0, w * p, 0).sum()
    assert (en.double() - entropy).abs().max().item() <= 2 * tol(0) * (1 + entropy), (en, entropy)
    for r in range(N):
        assert np.array_equal(ids[r].cpu().numpy(), order)
    return lp, en, ids, tops


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 10.0, 2.0 ** 100])
def test_a_forced_token(dtype, scale):
    """One column at the largest finite value: its probability is 1. (Its weight is 2^d, d the distance of scale log2(e)
    times it from the next whole number, within 4 u for the exponential and u for d; log2 of that 2 u: 8 u with the last
    product's, and as much for the entropy, which is log2 s - t / s of the same d.)"""
    for N, V in SIZES:
        for at in (0, V // 2, V - 1):
            x = logits(dtype, 1, V, seed=5).expand(N, V).contiguous()
            x[:, at] = torch.finfo(TYPES[dtype]).max
            lp, en, ids, _ = run_overflowing(x, [at] * N, 5, scale)
            assert max(lp.abs().max().item(), en.abs().max().item()) <= 8 * 2.0 ** -24 and (ids[:, 0] == at).all()
            run_overflowing(x, [(at + 9) % V] * N, 5, scale)


@pytest.mark.parametrize("order", ["masked first", "masked last", "masked by turns", "rising", "falling", "segments"])
@pytest.mark.parametrize("scale", [1.0, 1e4])
def test_rows_that_change_between_near_and_far(order, scale):
    """Parts of a row at the lowest value, ordinary ones, and ladders through every size."""
    for N, V in SIZES:
        i = torch.arange(V)
        low = torch.finfo(torch.float32).min
        x = 3 * torch.randn(V, generator=torch.Generator().manual_seed(9))
        if order == "masked first":
            x[:V // 2] = low
        elif order == "masked last":
            x[V // 2:] = low
        elif order == "masked by turns":
            x[(i // 1500) % 2 == 0] = low
        elif order == "segments":
            x[(i // 9000) % 3 != 1] = low
        else:
            ladder = torch.sign(i - V / 2) * 2.0 ** ((i - V / 2).abs() * (125 / V))        # (to 2^62)
            x = (ladder if order == "rising" else -ladder).float()
        run_overflowing(x.expand(N, V).contiguous().cuda(), [V // 3] * N, 5, scale)


def test_infinities_and_nan_beside_far_logits():
    for N, V in SIZES[:3]:
        x = torch.full((N, V), torch.finfo(torch.float32).min, device="cuda")
        x[:, :300] = -math.inf
        x[0, V // 2] = math.nan
        x[1, V // 2] = math.inf
        if N > 2:
            x[2] = -math.inf
        run(x, [400] * N, 5, rows=range(min(N, 4)))
