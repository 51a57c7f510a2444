"""Host-side tests of attention of chunks, rotary positions and log probabilities (include/wbserve.h):
workspace sizes, refusals, the split of the work in whole numbers, and the oracle's definitions by hand. No
call here launches work."""
import ctypes
import math

import numpy as np
import pytest

import linear_attn_decode_amd as wb
from linear_attn_decode_amd import serve
from oracle import serving as O

P = ctypes.c_void_p
OK, EINVAL, ESIZE, EUNSUPPORTED, EALIGN = 0, -1, -2, -3, -5
A = 0x100000            # an address that is never used: every call here is refused before, or has nothing to do
B = 0x200000


@pytest.fixture(scope="module")
def lib():
    h = ctypes.CDLL(wb.LIB_PATH)
    for name, (res, args) in wb.SERVE_SIGNATURES.items():
        fn = getattr(h, name)
        fn.restype, fn.argtypes = res, args
    return h


def cache(**kw):
    f = dict(k=A, v=A, k_scale=None, v_scale=None, pages=10, page=16, H=4, D=128, dtype=serve.BF16)
    f.update(kw)
    return wb.KVCacheDesc(*(f[n] for n, _ in wb.KVCacheDesc._fields_))


def chunk(lib, c, q=A, q_row=1024, q_head=128, q_dtype=serve.BF16, N=5, R=2, Hq=8, table=A, width=8, lens=A, starts=A, scale=1.0,
          window=0, o=B, lse=None, work=None, work_bytes=0):
    return lib.kv_attend_chunk(c, q, q_row, q_head, q_dtype, N, R, Hq, table, width, lens, starts, scale, window, o, lse, work,
                               work_bytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(pages=0), EINVAL), (dict(H=0), EINVAL), (dict(dtype=serve.F32), EINVAL),
    (dict(dtype=serve.E4M3), EINVAL), (dict(k_scale=A, v_scale=A), EINVAL), (dict(page=4), EUNSUPPORTED), (dict(page=24), EUNSUPPORTED),
    (dict(page=8192), EUNSUPPORTED), (dict(D=96), EUNSUPPORTED), (dict(H=5000), EUNSUPPORTED), (dict(pages=1 << 28), EUNSUPPORTED),
    (dict(v=A + 8), EALIGN)])
def test_bad_caches_are_refused(lib, bad, code):
    n = ctypes.c_size_t()
    assert lib.kv_attend_chunk_work(cache(**bad), 5, 2, 8, 8, n) == code
    assert chunk(lib, cache(**bad)) == code


def test_chunk_refusals(lib):
    n = ctypes.c_size_t()
    assert lib.kv_attend_chunk_work(cache(), 5, 2, 8, 8, n) == OK and n.value == 0       # 128 tokens: nothing is split
    assert lib.kv_attend_chunk_work(cache(), 5, 2, 8, 9, n) == OK and n.value > 0
    assert lib.kv_attend_chunk_work(cache(), 5, 2, 8, 9, None) == EINVAL
    assert chunk(lib, cache(), N=0) == OK
    assert chunk(lib, cache(), N=0, q=None, table=None, lens=None, starts=None, o=None, width=9) == OK
    for kw, code in [(dict(N=-1), EINVAL), (dict(R=0), EINVAL), (dict(R=65537), EUNSUPPORTED), (dict(Hq=0), EINVAL), (dict(Hq=9), EINVAL),
                     (dict(Hq=8192), EUNSUPPORTED), (dict(N=1 << 28), EUNSUPPORTED), (dict(width=0), EINVAL),
                     (dict(width=(1 << 26) + 1), EUNSUPPORTED), (dict(q=None), EINVAL), (dict(table=None), EINVAL), (dict(lens=None), EINVAL),
                     (dict(starts=None), EINVAL), (dict(o=None), EINVAL), (dict(window=-1), EINVAL), (dict(q_dtype=serve.F32), EINVAL),
                     (dict(q_dtype=serve.E4M3), EINVAL), (dict(q_dtype=9), EINVAL), (dict(q_dtype=serve.F16), EUNSUPPORTED),
                     (dict(q=A + 2), EALIGN), (dict(q_row=1020), EALIGN), (dict(q_head=130), EALIGN), (dict(o=B + 8), EALIGN),
                     (dict(table=A + 2), EALIGN), (dict(lens=A + 1), EALIGN), (dict(starts=A + 2), EALIGN), (dict(lse=A + 2), EALIGN),
                     (dict(o=A), EINVAL), (dict(width=9), EINVAL), (dict(width=9, work=A, work_bytes=n.value - 1), ESIZE),
                     (dict(width=9, work=A + 8, work_bytes=n.value), EALIGN), (dict(R=65), EINVAL),
                     (dict(R=65, work=A, work_bytes=67 * 8 - 1), ESIZE)]:
        assert chunk(lib, cache(), **kw) == code, kw
    assert chunk(lib, cache(dtype=serve.E4M3, k_scale=A, v_scale=A), q_dtype=serve.E4M3) == EINVAL


TARGET = 512            # parts that all tiles are cut into


def plan(N, R, Hq, H, D, page, width):
    """(Tokens of a block of rows, blocks of a key-value head's query heads, tokens of a key tile, slots)."""
    G = Hq // H
    heads, tile = min(G, 128), 32 if D == 256 else 64
    tokens, head_blocks, least = 128 // heads, -(-G // heads), 128 // tile
    blocks = min(N, N // tokens + R) * H * head_blocks
    tiles = -(-width * page // tile)
    return tokens, head_blocks, tile, min(blocks * -(-tiles // least), 2 * TARGET) if tiles > least else 0


@pytest.mark.parametrize("N,R,Hq,H,D,page,width", [(5, 2, 8, 4, 128, 16, 17), (8192, 1, 32, 8, 128, 64, 128), (64, 16, 40, 2, 64, 8, 1000),
                                                   (300, 300, 8, 8, 256, 16, 3), (7, 65, 300, 1, 256, 4096, 40), (1, 1, 1, 1, 64, 8, 1)])
def test_chunk_workspace(lib, N, R, Hq, H, D, page, width):
    """Sums of 128 rows for each part of a split block, their maximum and weight sum; of more than 64 requests the parts
    before each."""
    n = ctypes.c_size_t()
    assert lib.kv_attend_chunk_work(cache(H=H, D=D, page=page), N, R, Hq, width, n) == OK
    assert n.value == plan(N, R, Hq, H, D, page, width)[3] * 128 * (4 * D + 8) + (8 * (R + 2) if R > 64 else 0)


@pytest.mark.parametrize("seed", range(40))
def test_parts_stay_within_the_slots(seed):
    """Parts of t key tiles at most, t = max(128 tokens, all tiles / target): those of split blocks have slots, all have workgroups,
    and every tile of a block is in one part."""
    rng = np.random.default_rng(seed)
    H, G = int(rng.integers(1, 9)), int(rng.integers(1, 200))
    D, page, width = int(rng.choice([64, 256])), 16, int(rng.integers(1, 3000))
    R = int(rng.integers(1, 100))
    m = rng.integers(0, int(rng.choice([2, 9, 700])), R)
    n = np.minimum(m + rng.integers(0, width * page, R), np.maximum(width * page, m))
    m = np.where(n > width * page, 0, m)
    n = np.minimum(n, width * page)
    N, window = int(m.sum()), int(rng.choice([0, 0, 1, 100, 5000]))
    if N == 0:
        return
    tokens, head_blocks, tile, slots = plan(N, R, H * G, H, D, page, width)
    per_block = H * head_blocks
    span = -(-n // tile)
    if window:
        span = np.minimum(span, (window + tokens + 2 * tile - 3) // tile)
    span = np.maximum(span, 1)
    blocks = -(-m // tokens)
    most = max(128 // tile, -(-int((blocks * span).sum()) * per_block // TARGET))
    parts = -(-span // most)
    total, split = int((blocks * parts).sum()) * per_block, int((blocks * parts)[parts > 1].sum()) * per_block
    groups = min(N, N // tokens + R) * per_block + (TARGET if slots else 0)
    assert split <= slots and total <= groups, (split, slots, total, groups)
    for r in range(R):
        for b in range(int(blocks[r])):
            t0, t1, past = b * tokens, min((b + 1) * tokens, int(m[r])), int(n[r] - m[r])
            lo, hi = max(past + t0 - window + 1, 0) // tile if window else 0, -(-(past + t1) // tile)
            assert hi - lo <= span[r]
            ends = [lo + (hi - lo) * p // int(parts[r]) for p in range(int(parts[r]) + 1)]
            assert ends[0] == lo and ends[-1] == hi and all(x <= y for x, y in zip(ends, ends[1:]))


def heads(**kw):
    f = dict(x=A, out=A, weight=None, row=1024, head=128, out_row=1024, out_head=128, H=8, reserved=0)
    f.update(kw)
    return wb.HeadsDesc(*(f[n] for n, _ in wb.HeadsDesc._fields_))


def test_rotate_refusals(lib):
    def call(q=None, k=None, dtype=serve.BF16, N=3, D=128, positions=A, wide=0, freqs=A, rot=128, interleaved=0, magnitude=1.0, eps=1e-6):
        return lib.qk_rotate(heads() if q is None else q, k, dtype, N, D, positions, wide, freqs, rot, interleaved, magnitude, eps, None)
    nothing = heads(x=None, out=None)
    assert call(N=0) == OK and call(q=nothing, k=nothing, N=0, positions=None, freqs=None) == OK
    assert lib.qk_rotate(None, None, serve.BF16, 3, 128, A, 0, A, 128, 0, 1.0, 1e-6, None) == EINVAL
    for kw, code in [(dict(N=-1), EINVAL), (dict(D=0, rot=0), EINVAL), (dict(rot=-2), EINVAL), (dict(rot=130), EINVAL), (dict(rot=3), EINVAL),
                     (dict(dtype=serve.E4M3), EINVAL), (dict(dtype=9), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=math.nan), EINVAL),
                     (dict(magnitude=math.nan), EINVAL), (dict(D=1025, q=heads(head=1025, out_head=1025, row=8200, out_row=8200)), EUNSUPPORTED),
                     (dict(positions=None), EINVAL), (dict(freqs=None), EINVAL), (dict(freqs=A + 4), EALIGN),
                     (dict(positions=A + 2), EALIGN), (dict(positions=A + 4, wide=1), EALIGN)]:
        assert call(**kw) == code, kw
    for kw, code in [(dict(x=None), EINVAL), (dict(out=None), EINVAL), (dict(H=0), EINVAL), (dict(H=4097, row=1 << 20, out_row=1 << 20), EUNSUPPORTED),
                     (dict(out_row=1032), EINVAL), (dict(out_head=136, row=2048, out_row=2048), EINVAL),                 # in place: the same strides
                     (dict(out=B, out_head=64), EINVAL), (dict(out=B, out_row=64), EINVAL), (dict(out=B, out_row=512), EINVAL),
                     (dict(out=B, out_row=128, out_head=256), EINVAL), (dict(weight=A), EINVAL), (dict(out=B, weight=B), EINVAL),
                     (dict(x=B + 1), EALIGN), (dict(out=B + 1), EALIGN), (dict(weight=B + 1), EALIGN)]:
        assert call(q=heads(**kw)) == code, kw
        assert call(q=heads(x=4 * A, out=5 * A), k=heads(**kw)) == code, kw
    # keys and queries that are one another
    assert call(q=heads(), k=heads()) == EINVAL and call(q=heads(x=B), k=heads()) == EINVAL and call(q=heads(out=B), k=heads(x=B, out=4 * A)) == EINVAL
    assert call(q=heads(x=A + 2, out=B), dtype=serve.F32) == EALIGN


def test_logprob_refusals(lib):
    n = ctypes.c_size_t()
    assert lib.token_logprobs_work(0, 9, 0, n) == OK and n.value == 0
    assert lib.token_logprobs_work(5000, 151001, 20, n) == OK and n.value == 0           # rows enough for every compute unit
    assert lib.token_logprobs_work(1, 128000, 20, n) == OK and n.value > 0
    assert lib.token_logprobs_work(1, 128000, 20, None) == EINVAL
    for N, V, K, code in [(-1, 9, 0, EINVAL), (1, 0, 0, EINVAL), (1, 9, -1, EINVAL), (1, 9, 10, EINVAL), (1, (1 << 24) + 1, 0, EUNSUPPORTED),
                          (1, 900, 65, EUNSUPPORTED)]:
        assert lib.token_logprobs_work(N, V, K, n) == code

    def call(logits=A, row=900, dtype=serve.F32, N=3, V=900, tokens=A, wide=0, scale=1.0, logprob=B, entropy=None, K=0, ids=None, tops=None,
             work=None, work_bytes=0):
        return lib.token_logprobs(logits, row, dtype, N, V, tokens, wide, scale, logprob, entropy, K, ids, tops, work, work_bytes, None)
    assert call(N=0, logits=None, tokens=None, logprob=None) == OK
    big = dict(N=1, V=128000, row=128000, K=20, ids=A, tops=A)
    assert lib.token_logprobs_work(1, 128000, 20, n) == OK
    for kw, code in [(dict(N=-1), EINVAL), (dict(V=0), EINVAL), (dict(K=901, ids=A, tops=A), EINVAL), (dict(K=65, ids=A, tops=A), EUNSUPPORTED),
                     (dict(dtype=serve.E4M3), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=math.nan), EINVAL),
                     (dict(scale=2.0 ** -101), EUNSUPPORTED), (dict(scale=2.0 ** 101), EUNSUPPORTED), (dict(scale=math.inf), EUNSUPPORTED),
                     (dict(logits=None), EINVAL), (dict(tokens=None), EINVAL), (dict(logprob=None), EINVAL), (dict(K=3, ids=A), EINVAL),
                     (dict(K=3, tops=A), EINVAL), (dict(row=899), EINVAL), (dict(logits=A + 2), EALIGN), (dict(tokens=A + 2), EALIGN),
                     (dict(tokens=A + 4, wide=1), EALIGN), (dict(logprob=B + 1), EALIGN), (dict(entropy=B + 2), EALIGN),
                     (dict(K=3, ids=A + 1, tops=A), EALIGN), (dict(K=3, ids=A, tops=A + 2), EALIGN), (big, EINVAL),
                     (dict(work=A, work_bytes=n.value - 1, **big), ESIZE), (dict(work=A + 8, work_bytes=n.value, **big), EALIGN)]:
        assert call(**kw) == code, kw


@pytest.mark.parametrize("K", [1, 2, 5, 16, 31, 32, 33, 50, 64])
def test_logprob_segments_fit_their_memory(lib, K):
    """From the workspace's size (sums and K keys a segment, a counter a row): segments a lane each, their keys in one list
    of 4096, and 512 groups of 1024 columns in a segment at most, or of 512 where K groups of 1024 have more than 4096
    vectors; from any alignment of the row on."""
    n = ctypes.c_size_t()
    most = 2 ** 24 - 8 * (K > 32)
    assert lib.token_logprobs_work(1, most + 1, K, n) == EUNSUPPORTED
    for V in [most, most - 1, 2 ** 24 - 600, 2 ** 23 + 1, 2 ** 21 + 5, 2 ** 19 + 1, 2 ** 18, 151001, 128000, 20000, 9000, 700, K]:
        for N in (1, 2, 3, 7, 40, 255, 256, 257, 5000):
            if lib.token_logprobs_work(N, V, K, n) == OK:
                segments = (n.value // N // 8 - 1) // (2 + K) if n.value else 1
                assert n.value in (0, 8 * N * (segments * (2 + K) + 1)) and segments <= 64 and segments * K <= 4096
                columns = 1024 if K <= 32 else 512
                assert K * columns // 8 <= 4096
                chunks = -(-(V + 7) // columns)
                assert -(-chunks // segments) <= 512, (N, V, K, segments)
            else:
                assert V > most


def test_binding_refuses_cpu_tensors_and_sizes_past_32_bits():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    with pytest.raises(ValueError, match="k_cache: expected a tensor on the GPU"):
        wb.kv_attend_chunk(z(1, 1, 64), z(1, 1, 16, 64), z(1, 1, 16, 64), z(1, 1), z(1), z(2), z(1, 1, 64))
    with pytest.raises(ValueError, match="q: expected a tensor on the GPU"):
        wb.qk_rotate(z(1, 1, 64), None, z(1), z(32))
    with pytest.raises(ValueError, match="logits: expected a tensor on the GPU"):
        wb.token_logprobs(z(1, 9), z(1), z(1))


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=-2), dict(rot=8, base=0.0), dict(rot=8, base=math.nan), dict(rot=8, factor=0.0),
                                dict(rot=8, context=-1), dict(rot=8, context=10, slow=2.0, fast=2.0), dict(rot=8, context=10, slow=-1.0)])
def test_frequencies_out_of_range(kw):
    with pytest.raises(ValueError, match="are out of range"):
        wb.rotary_frequencies(device="cpu", **kw)


def test_frequencies_by_hand():
    f = wb.rotary_frequencies(4, base=100.0, device="cpu")
    assert f.tolist() == [1.0, 0.1] and len(wb.rotary_frequencies(0, device="cpu")) == 0
    assert wb.rotary_frequencies(4, base=100.0, factor=4.0, device="cpu").tolist() == [0.25, 0.025]
    # 2 pi * 10 positions: the pairs make 10 turns and 1: the first stays, the second is divided
    f = wb.rotary_frequencies(4, base=100.0, factor=4.0, context=round(20 * math.pi), slow=1.1, fast=9.0, device="cpu").numpy()
    assert np.allclose(f, [1.0, 0.025], rtol=1e-12)
    # half way between: half of each
    f = wb.rotary_frequencies(2, factor=4.0, context=63, slow=0.0, fast=2 * 63 / (2 * math.pi), device="cpu").numpy()
    assert np.allclose(f, [0.5 + 0.5 / 4], rtol=1e-12)


def test_oracle_attend_chunk_by_hand():
    v = np.array([[[1.0, 0.0]], [[0.0, 2.0]], [[5.0, 5.0]]])
    q, k = np.ones((2, 1, 2)), np.zeros((3, 1, 2))
    o, lse, _, _ = O.attend_chunk(q, k, v, 1.0)          # equal scores: means of the values up to each token
    assert np.allclose(o[:, 0], [[0.5, 1.0], [2.0, 7 / 3]]) and np.allclose(lse[:, 0], np.log([2, 3]))
    o, lse, _, _ = O.attend_chunk(q, k, v, 1.0, window=1)
    assert np.allclose(o[:, 0], v[1:, 0]) and np.allclose(lse, 0.0)
    # what one token sees is what attend gives for it, heads sharing a key-value head
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    for window in (0, 4):
        o, lse, W, size = O.attend_chunk(q, k, v, 0.3, window)
        for i in range(3):
            one = O.attend(q[i], k[:7 + i], v[:7 + i], 0.3, window)
            for a, b in zip((o, lse, W, size), one):
                assert np.allclose(a[i], b, rtol=1e-13)


def test_oracle_rotate_by_hand():
    x = np.array([[[1.0, 0.0, 3.0, 7.0]]])
    y, _ = O.rotate(x, None, 0.0, [1], [math.pi / 2], False, 2.0)      # a quarter turn of (x0, x1), twice as long
    assert np.allclose(y, [[[0.0, 2.0, 3.0, 7.0]]])
    y, _ = O.rotate(x, None, 0.0, [1], [math.pi / 2, 0.0], False, 1.0)  # halves: (x0, x2), (x1, x3)
    assert np.allclose(y, [[[-3.0, 0.0, 1.0, 7.0]]])
    y, _ = O.rotate(x, None, 0.0, [1], [math.pi / 2, 0.0], True, 1.0)   # neighbours: (x0, x1), (x2, x3)
    assert np.allclose(y, [[[0.0, 1.0, 3.0, 7.0]]])
    y, _ = O.rotate(np.array([[[3.0, 4.0]]]), np.array([1.0, 2.0]), 0.0, [0], [], False, 1.0)
    assert np.allclose(y, [[[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]]])
    assert (O.rotate(np.zeros((1, 1, 2)), np.ones(2), 0.0, [0], [], False, 1.0)[0] == 0).all()


def test_oracle_logprobs_by_hand():
    lp, en, order, p = O.logprobs(np.log([1.0, 2.0, 4.0, 1.0]), 1, 4)
    assert np.isclose(lp, math.log(0.25)) and order.tolist() == [2, 1, 0, 3] and np.allclose(p, np.log([0.5, 0.25, 0.125, 0.125]))
    assert np.isclose(en, 0.5 * math.log(2) + 0.25 * math.log(4) + 0.25 * math.log(8))
    lp, en, order, p = O.logprobs([0.0, -math.inf, 0.0], 1, 3, scale=5.0)
    assert lp == -math.inf and np.isclose(en, math.log(2)) and order.tolist() == [0, 2, 1] and p[2] == -math.inf
    assert np.isnan(O.logprobs([0.0, 1.0], -1, 1)[0]) and np.isnan(O.logprobs([0.0, math.nan], 0, 2)[1])
    assert O.logprobs([0.0, math.nan], 0, 2)[2].tolist() == [0, 1]
