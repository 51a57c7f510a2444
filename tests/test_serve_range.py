"""The serving operators' binding at the ends of its arguments' ranges. No call here launches work."""
import ctypes

import pytest

import linear_attn_decode_amd as wb
from linear_attn_decode_amd import serve

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("group", [2 ** 32, 2 ** 32 + 128, 128 - 2 ** 32, -2 ** 31, 2 ** 31, 2 ** 63 + 128])
def test_groups_past_32_bits_are_refused(group):
    """The library takes 32 bits: 2^32 + 128 would arrive as 128, and a scale for each 128
    columns be written where the binding has checked for one a row."""
    assert ctypes.c_int(2 ** 32 + 128).value == 128 and ctypes.c_int(128 - 2 ** 32).value == 128
    x = torch.zeros(2, 1024)
    with pytest.raises(ValueError, match="group: .* is out of range"):
        wb.norm_quant(x, None, x.to(torch.float8_e4m3fn), torch.zeros(2, 1), group=group)


@pytest.mark.parametrize("page", [2 ** 32 + 16, 16 - 2 ** 32, -2 ** 31, 2 ** 31])
def test_pages_past_32_bits_are_refused(page):
    n, one, table = (torch.zeros(s, dtype=torch.int32) for s in (1, 1, (1, 1)))
    with pytest.raises(ValueError, match="page: .* is out of range"):
        wb.plan_pages(n, n, table, n, one, page, torch.zeros(1, dtype=torch.int64), torch.zeros(2, dtype=torch.int32), one)
    with pytest.raises(ValueError, match="page: .* is out of range"):
        wb.release_pages(n, n, table, n, one, page, one)


def test_attention_into_its_own_query_is_refused():
    """Parts of a split request would read the query where another workgroup has stored the row.
    (The address is never used: the call is refused behind every other check.)"""
    h = ctypes.CDLL(wb.LIB_PATH)
    h.kv_attend.restype, h.kv_attend.argtypes = wb.SERVE_SIGNATURES["kv_attend"]
    A = 0x100000
    c = wb.KVCacheDesc(A, A, None, None, 10, 16, 4, 128, serve.BF16)
    assert h.kv_attend(c, A, 1024, 128, serve.BF16, 2, 8, A, 8, A, 1.0, 0, A, None, None, 0, None) == -1
