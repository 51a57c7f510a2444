"""The log-sum-exp of kv_attend_chunk (include/wbserve.h) over flat scores of 0: log n, within four of its last places (three
for the device's float32 logarithm, what OpenCL asks of it, one for the rest; the sum of n weights of 1 is exact), and 0 for
a single token."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("qt", ["bf16", "f16"])
@pytest.mark.parametrize("lens", [list(range(1, 60)), [100, 640, 5000, 20000]])
def test_flat_scores(qt, lens):
    """Requests of one new token each; the long ones are split and joined."""
    import linear_attn_decode_amd as wb
    print(f"[case] flat q={qt} lens={lens[:4]}", flush=True)
    page, D = 16, 64
    k = torch.zeros((1250, 1, page, D), dtype=TYPES[qt], device="cuda")
    q = torch.ones((len(lens), 1, D), dtype=TYPES[qt], device="cuda")
    table = torch.arange(1250, dtype=torch.int32).expand(len(lens), -1).contiguous().cuda()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    lse = torch.empty((len(lens), 1), device="cuda")
    wb.kv_attend_chunk(q, k, k.clone(), table, i32(lens), i32(list(range(len(lens) + 1))), torch.empty_like(q), lse=lse)
    torch.cuda.synchronize()
    want = np.log(np.asarray(lens, np.float64))
    place = np.spacing(want.astype(np.float32)).astype(np.float64)
    err = np.abs(lse[:, 0].double().cpu().numpy() - want)
    assert (err <= 4 * place).all(), (err / place).max()
    assert lens[0] != 1 or lse[0, 0].item() == 0
