"""Host-side tests of WB_ONE_LIMB (include/wbserve.h): the flag is part of q_dtype, and leaves every refusal as it is."""
import ctypes
import re
from pathlib import Path

import pytest

import linear_attn_decode_amd as wb
from linear_attn_decode_amd import serve
from tests.test_serve_prompt_abi import A, B, EALIGN, EINVAL, EUNSUPPORTED, OK, cache, chunk, lib  # noqa: F401


def test_the_bindings_value_is_the_headers():
    text = (Path(wb.__file__).parent.parent / "include" / "wbserve.h").read_text()
    assert int(re.search(r"#define WB_ONE_LIMB (\d+)", text)[1]) == serve.ONE_LIMB


@pytest.mark.parametrize("q_dtype,code", [(serve.BF16, EALIGN), (serve.F16, EUNSUPPORTED), (serve.F32, EINVAL), (serve.E4M3, EINVAL),
                                          (9, EINVAL), (-1, EINVAL), (512, EINVAL), (-256, EINVAL), (256, EINVAL)])
def test_refusals_with_the_flag(lib, q_dtype, code):  # noqa: F811
    """(A table that is not aligned: what is refused only behind the types.)"""
    flag = serve.ONE_LIMB if q_dtype in (serve.BF16, serve.F16, serve.F32, serve.E4M3, 9, 512) else 0
    if q_dtype == 256:                                          # the flag twice is another number
        flag = 256
    assert chunk(lib, cache(), q_dtype=q_dtype + flag, table=A + 2) == code
    assert chunk(lib, cache(), q_dtype=serve.BF16 + serve.ONE_LIMB, N=0) == OK
    scaled = cache(dtype=serve.E4M3, k_scale=A, v_scale=A)
    for q in (serve.BF16, serve.F16):
        assert chunk(lib, scaled, q_dtype=q + serve.ONE_LIMB, o=B + 8) == EALIGN


def test_workspaces_do_not_depend_on_it(lib):  # noqa: F811
    n = ctypes.c_size_t()
    assert lib.kv_attend_chunk_work(cache(), 5, 2, 8, 9, n) == OK
    assert chunk(lib, cache(), q_dtype=serve.BF16 + serve.ONE_LIMB, width=9, work=A, work_bytes=n.value - 1) == -2
