"""Host-side tests of the serving operators' C ABI (include/wbserve.h) and of the oracle's
8-bit format: exported symbols, workspace sizes, refusals. No call here launches work."""
import ctypes
import os
import re

import numpy as np
import pytest

import linear_attn_decode_amd as wb
from linear_attn_decode_amd import serve
from oracle import serving as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
OK, EINVAL, ESIZE, EUNSUPPORTED, EALIGN = 0, -1, -2, -3, -5
A = 0x100000            # an address that is never used: every call here is refused before


@pytest.fixture(scope="module")
def lib():
    h = ctypes.CDLL(wb.LIB_PATH)
    for name, (res, args) in wb.SERVE_SIGNATURES.items():
        fn = getattr(h, name)
        fn.restype, fn.argtypes = res, args
    return h


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "wbserve.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(wb.SERVE_SIGNATURES)
    h = ctypes.CDLL(wb.LIB_PATH)
    for n in names:
        assert hasattr(h, n), n


def cache(**kw):
    f = dict(k=A, v=A, k_scale=None, v_scale=None, pages=10, page=16, H=4, D=128, dtype=serve.BF16)
    f.update(kw)
    return wb.KVCacheDesc(*(f[n] for n, _ in wb.KVCacheDesc._fields_))


BAD_CACHES = [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(pages=0), EINVAL), (dict(H=0), EINVAL),
    (dict(dtype=serve.F32), EINVAL), (dict(dtype=7), EINVAL), (dict(dtype=serve.E4M3), EINVAL),
    (dict(k_scale=A, v_scale=A), EINVAL), (dict(dtype=serve.E4M3, k_scale=A), EINVAL),
    (dict(page=4), EUNSUPPORTED), (dict(page=24), EUNSUPPORTED), (dict(page=8192), EUNSUPPORTED),
    (dict(page=0), EUNSUPPORTED), (dict(page=-16), EUNSUPPORTED), (dict(D=96), EUNSUPPORTED), (dict(D=512), EUNSUPPORTED),
    (dict(pages=1 << 28), EUNSUPPORTED), (dict(H=5000), EUNSUPPORTED), (dict(k=A + 8), EALIGN),
]


def attend(lib, c, q=A, q_row=512, q_head=128, q_dtype=serve.BF16, R=2, Hq=8, table=A, width=8, lens=A, window=0, o=A,
           lse=None, work=None, work_bytes=0):
    return lib.kv_attend(c, q, q_row, q_head, q_dtype, R, Hq, table, width, lens, 1.0, window, o, lse, work, work_bytes, None)


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches_are_refused(lib, bad, code):
    n = ctypes.c_size_t()
    c = cache(**bad)
    assert lib.kv_attend_work(c, 2, 8, 8, n) == code
    assert attend(lib, c) == code
    assert lib.kv_append(c, A, A, 512, 512, serve.BF16, A, 3, None) == code


def test_attend_refusals(lib):
    n = ctypes.c_size_t()
    assert lib.kv_attend_work(cache(), 2, 8, 8, n) == OK and n.value == 0        # 128 tokens: nothing to join
    assert lib.kv_attend_work(cache(), 2, 8, 9, n) == OK and n.value > 0
    assert lib.kv_attend_work(cache(), 2, 8, 8, None) == EINVAL
    for kw, code in [(dict(R=0), EINVAL), (dict(R=-1), EINVAL), (dict(R=65537), EUNSUPPORTED), (dict(Hq=0), EINVAL),
                     (dict(Hq=9), EINVAL), (dict(Hq=8192), EUNSUPPORTED), (dict(width=0), EINVAL),
                     (dict(width=(1 << 26) + 1), EUNSUPPORTED), (dict(q=None), EINVAL), (dict(table=None), EINVAL),
                     (dict(lens=None), EINVAL), (dict(o=None), EINVAL), (dict(window=-1), EINVAL),
                     (dict(q_dtype=serve.F32), EINVAL), (dict(q_dtype=serve.F16), EUNSUPPORTED), (dict(q=A + 2), EALIGN),
                     (dict(q_row=500), EALIGN), (dict(q_head=130), EALIGN), (dict(o=A + 8), EALIGN),
                     (dict(table=A + 2), EALIGN), (dict(lens=A + 1), EALIGN), (dict(lse=A + 2), EALIGN),
                     (dict(width=9), EINVAL), (dict(width=9, work=A, work_bytes=n.value - 1), ESIZE),
                     (dict(width=9, work=A + 8, work_bytes=n.value), EALIGN)]:
        assert attend(lib, cache(), **kw) == code, kw
    e = cache(dtype=serve.E4M3, k_scale=A, v_scale=A)
    assert attend(lib, e, q_dtype=serve.E4M3) == EINVAL


@pytest.mark.parametrize("groups", [1, 2, 7, 256, 768, 1024])
@pytest.mark.parametrize("seed", range(6))
def test_attend_runs_and_segments(groups, seed):
    """The split along the cache, in whole numbers as the kernels take it: workgroup w of n
    takes units [total w // n, total (w + 1) // n); the workgroup of unit u is
    ((u + 1) n - 1) // total; every unit is in one run, an unfinished segment is its
    workgroup's first or last, and a request's block joins one segment per workgroup."""
    rng = np.random.default_rng(seed)
    blocks = int(rng.integers(1, 9))
    turns = rng.integers(1, 1 + 10 ** int(rng.integers(0, 4)), int(rng.integers(1, 40)))
    total = int(turns.sum()) * blocks
    n = min(total, groups)
    start = [total * w // n for w in range(n + 1)]
    assert all(b > a for a, b in zip(start, start[1:])) and start[0] == 0 and start[n] == total
    bounds = [0]
    for t in turns:
        bounds += [bounds[-1] + int(t) * (b + 1) for b in range(blocks)]
    for a, b in zip(bounds, bounds[1:]):
        w0, w1 = ((a + 1) * n - 1) // total, (b * n - 1) // total
        assert start[w0] <= a < start[w0 + 1] and start[w1] <= b - 1 < start[w1 + 1]
        for w in range(w0, w1 + 1):
            if w0 < w1:                                          # unfinished: first or last of w's run
                assert max(a, start[w]) == start[w] or min(b, start[w + 1]) == start[w + 1]
                assert w == w0 or start[w] > a                   # (slot 0 of every workgroup but the first)


def test_attend_workspace(lib):
    """Two segments of 16 rows of D sums, their maximum and weight sum for each workgroup,
    a first unit for each request and the end, a counter for each workgroup."""
    n = ctypes.c_size_t()
    for R, Hq, H, width, D, groups in ((1, 32, 8, 8192, 128, 256), (256, 32, 4, 512, 128, 256), (3, 40, 2, 9, 64, 3 * 2 * 2 * 2),
                                       (65536, 1, 1, 100, 64, 768), (2, 8, 8, 4096, 256, 256)):
        assert lib.kv_attend_work(cache(H=H, D=D), R, Hq, width, n) == OK
        blocks = H * -(-(Hq // H) // 16)
        groups = min(groups, R * blocks * -(-width * 16 // 128))
        assert n.value == groups * 2 * 16 * (4 * D + 8) + 8 * (R + 1) + 8 * groups


def test_append_refusals(lib):
    def call(c=cache(), k=A, v=A, k_row=512, v_row=512, src=serve.BF16, slots=A, N=3):
        return lib.kv_append(c, k, v, k_row, v_row, src, slots, N, None)
    e = cache(dtype=serve.E4M3, k_scale=A, v_scale=A)
    assert call(N=0) == OK and call(N=0, k=None, v=None, slots=None) == OK
    for kw, code in [(dict(N=-1), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(slots=None), EINVAL),
                     (dict(src=9), EINVAL), (dict(src=serve.F16), EUNSUPPORTED), (dict(src=serve.E4M3), EUNSUPPORTED),
                     (dict(c=e, src=serve.E4M3), EUNSUPPORTED), (dict(k_row=511), EINVAL), (dict(v_row=0), EINVAL),
                     (dict(k_row=516), EALIGN), (dict(N=1 << 30), EUNSUPPORTED), (dict(v=A + 4), EALIGN), (dict(slots=A + 4), EALIGN)]:
        assert call(**kw) == code, kw


def test_plan_and_release_refusals(lib):
    for in_place in (0, 1):
        assert lib.kv_plan_work(64, 64, in_place) == 0 and lib.kv_plan_work(5000, 64, in_place) == 5000
    assert lib.kv_plan_work(64, 1 << 20, 1) == 64 and lib.kv_plan_work(64, 1 << 20, 0) == 0

    def plan(lens=A, more=A, R=4, table=A, width=8, free=A, free_size=9, n_free=A, page=16, slots=A, n_slots=4, starts=A,
             lens_out=A, n_free_out=A, status=A, work=None):
        return lib.kv_plan_pages(lens, more, R, table, width, free, free_size, n_free, page, slots, n_slots, starts,
                                 lens_out, n_free_out, status, work, None)
    for name in ("lens", "more", "table", "n_free", "starts", "lens_out", "n_free_out", "status", "slots", "free"):
        assert plan(**{name: None}) == EINVAL, name
    for kw, code in [(dict(R=0), EINVAL), (dict(R=70000), EUNSUPPORTED), (dict(width=0), EINVAL), (dict(page=12), EUNSUPPORTED),
                     (dict(width=1 << 27), EUNSUPPORTED), (dict(n_slots=-1), EINVAL), (dict(n_slots=1 << 31), EUNSUPPORTED),
                     (dict(free_size=-1), EINVAL), (dict(slots=A + 8), EALIGN), (dict(lens=A + 1), EALIGN),
                     (dict(n_slots=1 << 20), EINVAL)]:
        assert plan(**kw) == code, kw

    def release(ended=A, lens=A, R=4, table=A, width=8, free=A, free_size=9, n_free=A, page=16, status=A):
        return lib.kv_release_pages(ended, lens, R, table, width, free, free_size, n_free, page, status, None)
    for name in ("ended", "lens", "table", "free", "n_free", "status"):
        assert release(**{name: None}) == EINVAL, name
    assert release(R=0) == EINVAL and release(page=100) == EUNSUPPORTED and release(lens=A + 2) == EALIGN


def test_norm_refusals(lib):
    def norm(x=A, x_row=256, residual=None, r_row=256, residual_out=None, ro_row=256, weight=None, dtype=serve.BF16, N=2,
             D=256, eps=1e-6, group=128, codes=A, c_row=256, scales=A):
        return lib.norm_quant(x, x_row, residual, r_row, residual_out, ro_row, weight, dtype, N, D, eps, group, codes, c_row,
                              scales, None)
    assert norm(N=0) == OK
    for kw, code in [(dict(x=None), EINVAL), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(N=-1), EINVAL),
                     (dict(D=0), EINVAL), (dict(dtype=serve.E4M3), EINVAL), (dict(residual=A), EINVAL),
                     (dict(residual_out=A), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
                     (dict(group=64), EUNSUPPORTED), (dict(group=-128), EUNSUPPORTED), (dict(D=65537, x_row=65537, c_row=65537), EUNSUPPORTED),
                     (dict(x_row=255), EINVAL), (dict(c_row=255), EINVAL), (dict(residual=A, residual_out=A, r_row=10), EINVAL),
                     (dict(residual=A, residual_out=A, ro_row=300), EINVAL), (dict(x=A + 1), EALIGN), (dict(weight=A + 1), EALIGN),
                     (dict(scales=A + 2), EALIGN), (dict(dtype=serve.F32, x=A + 2), EALIGN)]:
        assert norm(**kw) == code, kw


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    with pytest.raises(ValueError, match="x: expected a tensor on the GPU"):
        wb.norm_quant(z(2, 8), None, z(2, 8), z(2, 1))
    with pytest.raises(ValueError, match="k_cache: expected a tensor on the GPU"):
        wb.kv_attend(z(1, 1, 64), z(1, 1, 16, 64), z(1, 1, 16, 64), z(1, 1), z(1), z(1, 1, 64))
    with pytest.raises(ValueError, match="k_cache: expected a tensor on the GPU"):
        wb.kv_append(z(1, 1, 64), z(1, 1, 64), z(1, 1, 16, 64), z(1, 1, 16, 64), z(1))
    with pytest.raises(ValueError, match="lens: expected a tensor on the GPU"):
        wb.plan_pages(z(1), z(1), z(1, 1), z(1), z(1), 16, z(1), z(2), z(1))
    with pytest.raises(ValueError, match="lens: expected a tensor on the GPU"):
        wb.release_pages(z(1), z(1), z(1, 1), z(1), z(1), 16, z(1))


def test_oracle_e4m3_values():
    v = O.e4m3_values()
    assert np.nanmax(v) == 448.0 and np.isnan(v[127]) and np.isnan(v[255]) and v[1] == 2.0 ** -9 and v[0x38] == 1.0
    pos = v[:127]
    assert (np.diff(pos) > 0).all()
    # half a step around a value is half the distance to the next one, inside a binade
    for a, b in zip(pos[1:-1], pos[2:]):
        assert O.e4m3_half_step((a + b) / 2) == (b - a) / 2
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(t, v.astype(np.float32), equal_nan=True)


def test_oracle_plan_and_release_by_hand():
    table = np.full((3, 3), -1, np.int32)
    table[0, 0], table[2, 0] = 5, 6
    free = np.array([1, 2, 3, 4], np.int32)
    t, slots, starts, lens, n_free, status = O.plan([7, 0, 8], [3, 0, 1], table, free, 4, 8, 6)
    assert status == 0 and n_free == 2 and list(starts) == [0, 3, 3, 4] and list(lens) == [10, 0, 9]
    assert list(slots) == [5 * 8 + 7, 4 * 8, 4 * 8 + 1, 3 * 8, -1, -1]
    assert t[0].tolist() == [5, 4, -1] and t[2].tolist() == [6, 3, -1]
    lens, free, n_free, status = O.release([1, 0, 0], lens, t, free, n_free, 8)
    assert status == 0 and n_free == 4 and free.tolist() == [1, 2, 5, 4] and list(lens) == [0, 0, 9]
    assert O.plan([7], [3], table[:1], free, 0, 8, 6)[5] == 4 and O.plan([7], [30], table[:1], free, 4, 8, 6)[5] == 2
    assert O.plan([7], [3], table[:1], free, 4, 8, 2)[5] == 3 and O.plan([7], [-3], table[:1], free, 4, 8, 2)[5] == 1


def test_oracle_attend_by_hand():
    k = np.zeros((3, 1, 2))
    v = np.array([[[1.0, 0.0]], [[0.0, 2.0]], [[5.0, 5.0]]])
    q = np.array([[1.0, 1.0], [0.0, 0.0]])
    o, lse, _, _ = O.attend(q, k, v, 1.0)                # equal scores: the mean of the values
    assert np.allclose(o, [[2.0, 7 / 3]] * 2) and np.allclose(lse, np.log(3))
    o, lse, _, _ = O.attend(q, k, v, 1.0, window=1)
    assert np.allclose(o, 5.0) and np.allclose(lse, 0.0)
    o, lse, _, _ = O.attend(q, k[:0], v[:0], 1.0)
    assert (o == 0).all() and (lse == -np.inf).all()
