"""Which rows a request of kv_attend_chunk has when its starts decrease or leave [0, N] (include/wbserve.h): none, and nobody
else's are touched."""
import math

import numpy as np
import pytest

from tests.test_gpu_serve_chunk import check, rand, stored64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
N, LENS = 96, [40, 64, 50]


@pytest.mark.parametrize("starts,rows", [
    ([0, -5, 10, 20], {2: (10, 20)}),                     # the first ends, the second begins before row 0
    ([-5, 10, 20, 20], {1: (10, 20)}),
    ([-9, -5, -1, -1], {}),
    ([0, 30, 10, 10], {0: (0, 30)}),                      # the second decreases
    ([0, 10, N + 1, N + 1], {0: (0, 10)}),                # the second ends behind the last row
    ([0, 10, 20, N + 1], {0: (0, 10), 1: (10, 20)}),
    ([N + 5, N + 6, N, N], {}),                           # begins behind it
    ([2 ** 31 - 1, -2 ** 31, 5, 10], {2: (5, 10)}),
    ([7, 7, 7, 20], {2: (7, 20)}),                        # (rows before the first start are nobody's)
    ([N, N, N, N], {}),
    ([56, 96, 96, 96], {0: (56, 96)}),
])
@pytest.mark.parametrize("many", [False, True])
def test_rows_of_odd_starts(starts, rows, many):
    import linear_attn_decode_amd as wb
    print(f"[case] starts {starts} many={many}", flush=True)
    page, D, H, G, width = 16, 64, 2, 2, 4
    g = torch.Generator().manual_seed(2)
    k, v = (rand(g, 13, H, page, D, dtype="f16").cuda() for _ in range(2))
    q = rand(g, N, H * G, D, dtype="f16").cuda()
    lens, table = list(LENS), np.arange(12, dtype=np.int32).reshape(3, width)
    if many:                                                 # (past the lane count: requests without rows behind)
        starts, lens = starts + [starts[-1]] * 97, lens + [5] * 97
        table = np.concatenate([table, np.full((97, width), 12, np.int32)])
    i32 = lambda a: torch.tensor(np.asarray(a, np.int64).astype(np.int32)).cuda()
    o, lse = torch.full((N, H * G, D), 7.0, dtype=torch.float16, device="cuda"), torch.full((N, H * G), 7.0, device="cuda")
    wb.kv_attend_chunk(q, k, v, i32(table), i32(lens), i32(starts), o, lse=lse)
    torch.cuda.synchronize()
    left = torch.ones(N, dtype=torch.bool)
    for r, (a, b) in rows.items():
        check(o[a:b], lse[a:b], q[a:b], stored64(k, None), stored64(v, None), table[r:r + 1], [lens[r]], [0, b - a], page,
              1 / math.sqrt(D), 0, "f16", "f16")
        left[a:b] = False
    assert (o[left.cuda()] == 7).all() and (lse[left.cuda()] == 7).all()
