"""Page tables of kv_attend_chunk (include/wbserve.h) that a sliding window has left behind: pages that no row sees are given
back, and their entries hold no page. Tolerances as in tests/test_gpu_serve_chunk.py."""
import math

import numpy as np
import pytest

from tests.test_gpu_serve_chunk import check, make_table, rand, random_cache, stored64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def i32(a):
    return torch.tensor(np.asarray(a, np.int32)).cuda()


@pytest.mark.parametrize("kv,qt,D", [("bf16", "bf16", 64), ("f16", "f16", 128), ("e4m3", "bf16", 128), ("bf16", "bf16", 256), ("e4m3", "f16", 256)])
@pytest.mark.parametrize("page", [8, 16, 32, 64])
@pytest.mark.parametrize("window", [1, 7, 50, 129])
@pytest.mark.parametrize("gone", [-1, 2 ** 30])
def test_pages_before_every_window_are_not_looked_up(kv, qt, D, page, window, gone):
    import linear_attn_decode_amd as wb
    news, pasts, H, G = [1, 5, 1, 30, 150, 1], [200, 333, 7, 1000, 517, 4090], 2, 4
    lens, starts = [a + b for a, b in zip(news, pasts)], np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    print(f"[case] given back kv={kv} q={qt} D={D} page={page} window={window} id={gone}", flush=True)
    g, rng = torch.Generator().manual_seed(page + window), np.random.default_rng(window)
    pages = sum(-(-n // page) for n in lens) + 1
    table = make_table(rng, lens, page, pages, max(-(-n // page) for n in lens))
    k, ks = random_cache(g, pages, H, page, D, kv)
    v, vs = random_cache(g, pages, H, page, D, kv)
    q = rand(g, int(starts[-1]), H * G, D, dtype=qt).cuda()
    left = table.copy()
    for r, past in enumerate(pasts):
        left[r, :max(0, past + 1 - window) // page] = gone
    outs = []
    for t in (left, table):
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        wb.kv_attend_chunk(q, k, v, i32(t), i32(lens), i32(starts), o, window=window, lse=lse, k_scale=ks, v_scale=vs)
        torch.cuda.synchronize()
        outs.append((o, lse))
    check(*outs[0], q, stored64(k, ks), stored64(v, vs), table, lens, starts, page, 1 / math.sqrt(D), window, kv, qt)
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # the single tokens, by kv_attend
    one = [r for r, m in enumerate(news) if m == 1]
    rows = [int(starts[r]) for r in one]
    o1 = torch.empty((len(one), H * G, D), dtype=q.dtype, device="cuda")
    wb.kv_attend(q[rows].contiguous(), k, v, i32(left[one]), i32([lens[r] for r in one]), o1, window=window, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    assert torch.isfinite(o1).all() and torch.isfinite(outs[0][0]).all()


@pytest.mark.parametrize("page", [8, 64])
def test_a_page_that_a_window_reaches_by_one_token_is(page):
    import linear_attn_decode_amd as wb
    H, D, n, m, window = 1, 64, 640, 20, 100
    g = torch.Generator().manual_seed(page)
    k, v = (rand(g, n // page, H, page, D, dtype="bf16").cuda() for _ in range(2))
    q = rand(g, m, 2, D, dtype="bf16").cuda()
    table = np.arange(n // page, dtype=np.int32)[None].copy()
    first = n - m + 1 - window                               # of the first row's window: 521
    table[0, first // page] = -1
    o = torch.empty_like(q)
    wb.kv_attend_chunk(q, k, v, i32(table), i32([n]), i32([0, m]), o, window=window)
    torch.cuda.synchronize()
    sees = [p + 1 - window <= first // page * page + page - 1 for p in range(n - m, n)]
    assert sees[0] and torch.isnan(o[torch.tensor(sees).cuda()]).all()
