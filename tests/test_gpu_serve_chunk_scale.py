"""kv_attend_chunk (include/wbserve.h) at the ends of its scale."""
import math

import pytest

from tests.test_gpu_serve_chunk import TYPES, rand

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def i32(a):
    return torch.tensor(a, dtype=torch.int32).cuda()


@pytest.mark.parametrize("qt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("limbs", [1, 2])
def test_scale_zero_of_queries_that_are_not_finite(qt, D, limbs):
    """Scores of 0 for finite queries (o the mean of the values: their sum is exact, one rounding of the weights, 1, and one
    of o), NaN where a query holds an infinity or a NaN, as for kv_attend."""
    import linear_attn_decode_amd as wb
    print(f"[case] scale 0 q={qt} D={D} limbs={limbs}", flush=True)
    page, n, m = 16, 90, 40
    g = torch.Generator().manual_seed(1)
    k = rand(g, 6, 1, page, D, dtype=qt).cuda()
    v = (torch.randint(-8, 9, (6, 1, page, D), generator=g) / 8).to(TYPES[qt]).cuda()
    q = rand(g, m, 4, D, dtype=qt).cuda()
    bad = {(0, 1, 5): math.nan, (17, 0, 0): math.inf, (17, 3, D - 1): -math.inf, (39, 2, 33): math.nan}
    for (i, h, d), x in bad.items():
        q[i, h, d] = x
    o, lse = torch.empty_like(q), torch.empty((m, 4), device="cuda")
    table = i32([list(range(6))])
    wb.kv_attend_chunk(q, k, v, table, i32([n]), i32([0, m]), o, scale=0.0, lse=lse, limbs=limbs)
    one = torch.empty_like(q[-1:])
    wb.kv_attend(q[-1:].contiguous(), k, v, table, i32([n]), one, scale=0.0)
    torch.cuda.synchronize()
    holds = torch.zeros((m, 4), dtype=torch.bool)
    for i, h, _ in bad:
        holds[i, h] = True
    assert torch.isnan(o[holds.cuda()]).all() and torch.isnan(lse[holds.cuda()]).all()
    seen = torch.arange(n - m + 1, n + 1)
    mean = (v.double().cpu()[:, 0].reshape(-1, D).cumsum(0)[seen - 1] / seen[:, None])[:, None].expand(m, 4, D)
    half = torch.finfo(TYPES[qt]).eps / 2
    fine = ~holds
    assert ((o.double().cpu() - mean).abs() <= half * mean.abs() + 8 * 2.0 ** -24)[fine].all()
    # (a logarithm below 8, within two of its last places, 2^-21)
    assert ((lse.double().cpu() - seen.double().log()[:, None]).abs() <= 2.0 ** -20)[fine].all()
    assert torch.equal(torch.isnan(one[0]), torch.isnan(o[-1]))
