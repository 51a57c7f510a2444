// Attention of chunks of new tokens over a paged key-value cache (wbserve.h).
//
//   o_i = sum_t e^{s_it - m} v_t / sum_t e^{s_it - m},  s_it = scale q_i . k_t,  t <= position of i
//
// in one pass over the stored tokens with a running maximum. A key-value head's query heads read the same tokens, so a
// workgroup takes a block of 128 rows: the heads of as many neighbouring new tokens as give 128. Each of its 4 wavefronts
// has 32 of them, whose queries stay in registers; the tokens' keys and values go through LDS, which all rows share, in
// two tiles by turns: the next one's loads go from memory straight to LDS behind this one's products.
//
// Scores are taken transposed, K Q^T (32 x 32 x 16 products): a lane ends with 16 tokens of one row, whose maximum and sum
// need one exchange between two lanes, and whose weights are in place as an operand of V^T P^T, where a product's 16 tokens
// may come in any order as long as both operands agree. V's operand is read from LDS by transposing reads. Weights never
// leave registers, and the accumulators hold a row in a lane, so that its rescaling is one factor.
// The weights' reference moves only when a row's maximum has risen by more than 2^4 (kThreshold): 2^4 is far from the end
// of either type, and all tiles but a row's first few then go without rescaling the accumulators.
// Weights enter the second product as two limbs of 16 bits (2^-16 of each in bfloat16), so that the error of o is that of
// its own rounding. The second limb's products are a third of all: the caller may have one limb (half a step of each
// weight, 2^-8 in bfloat16: 1.1 to 1.45 times the error) and 8192-token prompts of heads of 128 in 543 us, not 721, 8-bit
// ones in 684, not 849, drafts in 93, not 97. A float16 query over an 8-bit cache always has two: bfloat16, which holds
// the values' scales, keeps 3 bits fewer than its output. Float16 weights are 2^11 of themselves
// (kShift; at most 2^15 with the lazy reference): what falls below its smallest step is 2^-36 of the largest. The sum of
// weights is taken in float32 of the weights before they are rounded, each tile's by itself, the tiles' with what their
// roundings leave.
//
// Prompts (8192 tokens, 32 / 8 heads of 128, bfloat16): 720 to 750 us, 1.10 to 1.15 PFLOP/s with the second limb's products,
// matrix cores busy 59 % of the cycles; a large library product reaches 1.16 to 1.23. With one limb they take 541 to 580 us
// (0.95 to 1.02 PFLOP/s), the matrix cores are busy 51 %, and what is not behind products limits them: the softmax 15 %, of
// which the exponentials 7, reading LDS 14 %, staging 16 % (each left out alone). Power limits both as well (clocks of 1.8
// to 2.05 GHz), but less than a plain product: over zeros the one-limb call takes 485 us, 12 % less, a library product
// 30 % less. Few rows over long caches are bound by reading the cache: 64 requests of 5 drafted tokens each, 367 MB, 97 us
// (3.8 TB/s), where the last parts end late and a second launch joins.
#include "serve_device.hpp"

namespace wb {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4, kThreads = 64 * kWaves, kRows = 32 * kWaves;
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------------------- where a workgroup works
// A request: its new tokens (rows first ..+m of q), stored tokens n; span: key tiles of a
// block of its rows at most. A bad length has n = 0 and one tile of which nothing is read.
struct Request {
    int first, m, n, blocks, span;
    bool bad;
};
__device__ __forceinline__ Request request_of(const ChunkArgs& A, int r) {
    Request q;
    const int s0 = A.starts[r], s1 = A.starts[r + 1], n = A.lens[r];
    q.first = s0;
    q.m = s0 < 0 || s1 > A.N || s1 < s0 ? 0 : s1 - s0;
    q.bad = n < q.m || n > (A.width << A.page_log2);
    q.n = q.bad ? 0 : n;
    q.blocks = (q.m + A.tokens - 1) / A.tokens;
    const int l2 = A.tile_log2, tile = 1 << l2;
    q.span = (q.n + tile - 1) >> l2;
    if (A.window) q.span = min(q.span, int((int64_t(A.window) + A.tokens + 2 * tile - 3) >> l2));
    q.span = max(q.span, 1);
    return q;
}

// Part `part` of `parts` of a block of rows (the block-th of request r, for head block hb of
// key-value head kvh). slot: of its sums in the workspace, slot0 its first part's.
struct Work {
    Request q;
    int r, block, kvh, hb, part, parts;
    int64_t slot, slot0;
};

// A part has at most this many key tiles: all tiles are cut into about A.target parts of at least A.part_tiles.
// (tiles: of all blocks of one head block)
__device__ __forceinline__ int part_limit(const ChunkArgs& A, int64_t tiles) {
    const int64_t all = tiles * (A.c.H * A.head_blocks);
    const int64_t most = max(int64_t(A.part_tiles), quotient64(all + A.target - 1, int64_t(A.target)));
    return int(min(most, int64_t(1) << 30));
}
// Parts of a request's blocks (lower half), and of those that are split (upper half)
__device__ __forceinline__ int64_t count_parts(const ChunkArgs& A, int blocks, int span, int most) {
    const int parts = blocks ? (span + most - 1) / most : 1;
    const int64_t n = int64_t(blocks) * (A.c.H * A.head_blocks) * parts;
    return n | (parts > 1 ? n : 0) << 32;
}

// The work of number `at`, among all parts, or among those of split blocks only. False: there are not so many. Every
// wavefront finds it for itself. Up to 64 requests are a lane's each, taken by their spans, long ones first, so that
// what is started last is short (64 ragged caches to 4096, 5 drafted tokens each: 97 us, 102 in the order they come; 16
// ragged prompts, 8-bit: 123 and 126; 64 caches of one length gain nothing by it, 43 and 38). Of
// more, a launch before this one has summed the parts (count_requests_kernel), and the sums are searched, 64 places a step.
template <bool SPLIT_ONLY>
__device__ __forceinline__ bool find_work(const ChunkArgs& A, int64_t at, Work& w) {
    const int lane = threadIdx.x & 63;
    const int per_block = A.c.H * A.head_blocks;
    auto key = [&](int64_t v) { return SPLIT_ONLY ? v >> 32 : v & 0xFFFFFFFF; };
    int64_t before;
    int most;
    if (A.R <= 64) {
        Request q{};
        if (lane < A.R) q = request_of(A, lane);
        most = part_limit(A, lane64(wave_scan(int64_t(q.blocks) * q.span), 63));
        int place = 0;
        for (int j = 0; j < A.R; ++j) {
            const int other = __builtin_amdgcn_readlane(q.span, j);
            place += other > q.span || (other == q.span && j < lane);
        }
        if (lane >= A.R) place = lane;
        const int id = __builtin_amdgcn_ds_permute(4 * place, lane);
        q.blocks = __builtin_amdgcn_ds_permute(4 * place, q.blocks);
        q.span = __builtin_amdgcn_ds_permute(4 * place, q.span);
        const int64_t mine = count_parts(A, q.blocks, q.span, most), upto = wave_scan(mine);
        if (key(lane64(upto, 63)) <= at) return false;
        const int who = __ffsll((unsigned long long)__ballot(key(upto) > at)) - 1;
        before = lane64(upto, who) - lane64(mine, who);
        w.r = __builtin_amdgcn_readlane(id, who);
    } else {
        if (key(A.before[A.R]) <= at) return false;
        most = int(A.before[A.R + 1]);
        int from = 0;                                        // the last request with no more than `at` parts before it
        for (int n = A.R, step; n > 1; n = min(step, A.R - from)) {
            step = (n + 63) / 64;
            const uint64_t upto = __ballot(lane * step < n && key(A.before[from + min(lane * step, n - 1)]) <= at);
            from += (63 - __builtin_clzll(upto | 1)) * step;
        }
        w.r = from;
        before = A.before[from];
    }
    auto parts_in = [&](const Request& q) { return (q.span + most - 1) / most; };
    w.r = __builtin_amdgcn_readfirstlane(min(w.r, A.R - 1));
    w.q = request_of(A, w.r);
    w.q.first = __builtin_amdgcn_readfirstlane(w.q.first);
    w.q.m = __builtin_amdgcn_readfirstlane(w.q.m);
    w.q.n = __builtin_amdgcn_readfirstlane(w.q.n);
    w.parts = __builtin_amdgcn_readfirstlane(parts_in(w.q));
    // blocks from the last (which has the most tokens before it) to the first, heads fastest
    const int64_t in_r = max(at - key(before), int64_t(0));
    const int64_t unit = in_r / per_block;
    const int head = int(in_r - unit * per_block);
    w.kvh = __builtin_amdgcn_readfirstlane(head / A.head_blocks);
    w.hb = __builtin_amdgcn_readfirstlane(head - w.kvh * A.head_blocks);
    const int64_t rev = unit / w.parts;
    w.part = __builtin_amdgcn_readfirstlane(int(unit - rev * w.parts));
    w.block = __builtin_amdgcn_readfirstlane(int(min(max(w.q.blocks - 1 - rev, int64_t(0)), int64_t(w.q.blocks - 1))));
    const int64_t split0 = before >> 32;
    w.slot0 = split0 + (rev * w.parts * per_block + head);
    w.slot = w.slot0 + int64_t(w.part) * per_block;
    return w.q.m > 0;
}

// before[r]: the parts of requests 0 .. r - 1; behind them, the key tiles of a part. (Of more than 64 requests: requests
// of 600 tokens, one of them new, 128 of them 64 us, 68 where each wavefront sums them for itself, 4096 1.67 ms and 5.35.)
constexpr int kCountThreads = 1024;
__global__ void __launch_bounds__(kCountThreads) count_requests_kernel(const ChunkArgs A) {
    __shared__ int64_t sums[kCountThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    auto scan = [&](int64_t v, int64_t& all) {                  // v summed over the threads up to this one
        const int64_t in = wave_scan(v);
        __syncthreads();
        if (lane == 63) sums[wave] = in;
        __syncthreads();
        int64_t below = 0;
        all = 0;
        for (int i = 0; i < kCountThreads / 64; ++i) {
            if (i < wave) below += sums[i];
            all += sums[i];
        }
        return below + in;
    };
    int64_t tiles = 0, all;
    for (int r = tid; r < A.R; r += kCountThreads) {
        const Request q = request_of(A, r);
        tiles += int64_t(q.blocks) * q.span;
    }
    scan(tiles, all);
    const int most = part_limit(A, all);
    int64_t done = 0;
    for (int base = 0; base < A.R; base += kCountThreads) {
        const int r = base + tid;
        Request q{};
        if (r < A.R) q = request_of(A, r);
        const int64_t mine = r < A.R ? count_parts(A, q.blocks, q.span, most) : 0, upto = scan(mine, all);
        if (r < A.R) A.before[r] = done + upto - mine;
        done += all;
    }
    if (tid == 0) {
        A.before[A.R] = done;
        A.before[A.R + 1] = most;
    }
}

// Key tiles [from, to) of a part
struct Tiles {
    int from, to;
};
__device__ __forceinline__ Tiles tiles_of(const ChunkArgs& A, const Request& q, int block, int part, int parts) {
    const int t0 = block * A.tokens, t1 = min(t0 + A.tokens, q.m);       // new tokens of the block
    const int past = q.n - q.m;
    const int lo = A.window ? max(past + t0 - A.window + 1, 0) >> A.tile_log2 : 0;
    const int hi = q.bad ? 0 : (past + t1 + (1 << A.tile_log2) - 1) >> A.tile_log2;
    const int n = max(hi - lo, 0);
    return Tiles{lo + int(int64_t(n) * part / parts), lo + int(int64_t(n) * (part + 1) / parts)};
}

// ---------------------------------------------------------------------------- operands
template <int T>
struct Mat32;
template <>
struct Mat32<WB_BF16> {
    static constexpr uint32_t kExponent = 0x7F80u;
    static __device__ __forceinline__ f32x16 mul(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    }
};
template <>
struct Mat32<WB_F16> {
    static constexpr uint32_t kExponent = 0x7C00u;
    static __device__ __forceinline__ f32x16 mul(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
    }
};
template <int T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {        // (one instruction)
    if constexpr (T == WB_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
}
template <int T>
__device__ __forceinline__ float low(uint32_t w) { return Elem<T>::get(uint16_t(w)); }
template <int T>
__device__ __forceinline__ float high(uint32_t w) { return Elem<T>::get(uint16_t(w >> 16)); }

// Two values (exact) of bytes 0, 1 or 2, 3 of four e4m3 codes
template <int T, bool HIGH>
__device__ __forceinline__ uint32_t e4m3_to2(uint32_t w) {
    if constexpr (T == WB_BF16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
    else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
}
template <int T>
__device__ __forceinline__ u32x4 e4m3_to8(u32x2 w) {
    return u32x4{e4m3_to2<T, false>(w[0]), e4m3_to2<T, true>(w[0]), e4m3_to2<T, false>(w[1]), e4m3_to2<T, true>(w[1])};
}

// Which of a word's two values are infinite or NaN (bits 15 and 31)
template <int T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    constexpr uint32_t e = Mat32<T>::kExponent * 0x10001u, one = T == WB_BF16 ? 0x00800080u : 0x04000400u;
    return ((w & e) + one) & 0x80008000u;
}

__device__ __forceinline__ s16x4 read_transposed(const uint8_t* at) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at);
}

// 16 bytes a lane from `base` + `off` bytes straight to LDS, the lane's after byte `to` of it (`base` and `to` are the same
// for all lanes). Written as assembly because behind the builtin the compiler lets every later read of LDS wait for
// all such loads: the next tile's would not stay in flight behind this one's products. It writes no register, so there
// is none for the compiler to use too early; lds_loads_wait() and a barrier come before the data is read.
__device__ __forceinline__ void lds_load16_async(const uint8_t* base, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : : "s"(to), "v"(off), "s"(base) : "memory", "m0");
}

// -infinity in place of x where d is negative. (A selection by sign bits: conditions in scalar registers, 32 of them
// at once, would push what the loop keeps there out.)
__device__ __forceinline__ float hide(float x, int d) {
    const uint32_t gone = uint32_t(d >> 31);
    return __uint_as_float((gone & 0xFF800000u) | (~gone & __float_as_uint(x)));
}

// 4 columns of a finished row, by 1 / its sum of weights, in two words of two
template <int QT>
__device__ __forceinline__ u32x2 scaled(f32x4 v, float by) {
    return u32x2{pack2<QT>(v[0] * by, v[1] * by), pack2<QT>(v[2] * by, v[3] * by)};
}

// Key tiles of 64 tokens, of 32 for heads of 256 columns: with 64 such a head's tiles, sums and scores fill a compute
// unit's memory and registers with one workgroup, whose matrix and vector units then take turns (8192-token prompts,
// 16 heads of 256, bfloat16: 856 us, 711 with two workgroups). Narrower heads have two either way, and the larger tile has
// fewer barriers and joins (8192-token prompts of heads of 128: 16 bits within 1 % of one another, 8-bit 849 us and 924
// with 32; ragged 8-bit 123 and 135; where rows are few and blocks equal, 32 is the faster: drafts 97 and 91).
constexpr int kWavesPerSimd = 2;
constexpr int tile_log2(int D) { return D <= 128 ? 6 : 5; }

// KV: the cache's type; QT: the type of q and o; D: columns; LIMBS: 16-bit values of a weight
template <int KV, int QT, int D, int LIMBS>
struct Chunk {
    static constexpr int ST = QT;                                    // operands of the scores
    static constexpr int VT = KV == WB_E4M3 ? WB_BF16 : KV;          // of the values
    static constexpr bool kTwoP = LIMBS == 2;
    static constexpr int KS = D / 16;                                // score products of 32 tokens
    static constexpr int DB = D / 32;                                // blocks of value columns
    static constexpr int CB = D / 64;                                // blocks of 64 columns
    static constexpr int kShift = VT == WB_F16 ? 11 : 0;             // weights enter as 2^kShift times their value
    static constexpr int kTile = 1 << tile_log2(D);
    static constexpr int NB = kTile / 32, TB = kTile / 8;            // its blocks of 32 tokens, of 8
    static constexpr int kTileBytes = kTile * D * 2;
    // A lane's sum of weights in LDS, where its two registers are one too many: 8192 tokens over 8-bit caches, heads of 64
    // 519 us (607 in registers, with two wavefronts a SIMD in place of three), of 256 948 (1038, more of them spilled);
    // heads of 128 and 16-bit caches are as fast or faster in registers (heads of 128 in float16 751, 771 in LDS)
    static constexpr bool kSumsInLds = KV == WB_E4M3 && D != 128;
};

// The kernel's arguments, read again here: held from its start, or through its loop, they would cost registers there
__device__ __forceinline__ const __attribute__((address_space(4))) ChunkArgs& arguments_again() {
    auto p = (const __attribute__((address_space(4))) ChunkArgs*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *p;
}

template <int KV, int QT, int D, int LIMBS>
__global__ void __launch_bounds__(kThreads, kWavesPerSimd) chunk_kernel(const ChunkArgs A) {
    using T = Chunk<KV, QT, D, LIMBS>;
    using S = Mat32<T::ST>;
    using V = Mat32<T::VT>;
    constexpr int KS = T::KS, DB = T::DB, CB = T::CB, kTile = T::kTile, NB = T::NB, TB = T::TB;
    constexpr bool E = KV == WB_E4M3;
    constexpr int kRowBytes = D * (E ? 1 : 2);
    constexpr float kThreshold = 4.f;            // (in powers of two; 0: an 8192-token prompt 747 us, not 721)
    __shared__ __attribute__((aligned(1024))) uint8_t stored[2][2][T::kTileBytes];        // [buffer][keys, values]
    __shared__ f32x4 scales[2][2][kTile / 4];
    __shared__ uint32_t strange_bits[kTile][DB];                     // of the tile's values: columns of each token
    __shared__ int strange, bad_page;

    Work w;
    if (!find_work<false>(A, A.launched + blockIdx.x, w)) return;
    const Tiles tiles = tiles_of(A, w.q, w.block, w.part, w.parts);
    if (w.parts > 1 && (tiles.from >= tiles.to || uint64_t(w.slot) >= uint64_t(A.slots))) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, col = lane & 31;
    if (tid == 0) strange = bad_page = 0;

    const auto& C = arguments_again();

    // The lane's row of q: row j of the block is head j % heads of token j / heads
    const int past = w.q.n - w.q.m, t0 = w.block * C.tokens, tokens = min(C.tokens, w.q.m - t0);
    int limit, lower;                   // tokens [lower, limit) are seen
    u32x4 qf[KS];
    {
        const int j = wave * 32 + col, token = j / C.heads, head = j - token * C.heads;
        const bool ok = token < tokens && head < min(C.heads, C.G - w.hb * C.heads);
        const int hq = w.kvh * C.G + w.hb * C.heads + head;
        limit = ok ? past + t0 + token + 1 : 0;
        lower = C.window ? max(limit - C.window, 0) : 0;
        const uint16_t* q = static_cast<const uint16_t*>(C.q) + (int64_t(w.q.first) + t0 + token) * C.q_row +
                            int64_t(hq) * C.q_head + 8 * h;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            qf[i] = u32x4{0, 0, 0, 0};
            if (ok && C.scale != 0.f) qf[i] = *reinterpret_cast<const u32x4*>(q + 16 * i);
            if (C.scale < 0.f) qf[i] ^= 0x80008000u;
        }
    }
    // (a scale of 0: scores of 0)
    const float mul = (C.scale == 0.f ? 1.f : fabsf(C.scale)) * kLog2e;
    // Tiles that some row of the wavefront sees, and those of which every row of the block sees all
    const int first_token = wave * 32 / C.heads, last_token = min((wave * 32 + 31) / C.heads, tokens - 1);
    int any_from = C.window ? max(past + t0 + first_token + 1 - C.window, 0) / kTile : 0;
    int any_to = first_token < tokens ? (past + t0 + last_token + kTile) / kTile : 0;
    const int whole_from = C.window ? (max(past + t0 + tokens - C.window, 0) + kTile - 1) / kTile : 0;
    const int whole_to = (past + t0 + 1) / kTile;
    const bool windowed = C.window != 0;

    f32x16 acc[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) acc[i] = f32x16{};
    float m = -INFINITY;
    __shared__ f32x2 lds_sums[T::kSumsInLds ? kThreads : 1];
    f32x2 register_sums;
    auto weights = [&]() -> f32x2& {                          // their sum, in two parts
        if constexpr (T::kSumsInLds) return lds_sums[tid];
        else return register_sums;
    };
    weights() = f32x2{0.f, 0.f};

    // ------------------------------------------------------------------ staging
    // A tile lies in LDS as blocks of 8 tokens by 64 columns, 1 KB each, block (c, g) at 1024 (8 c + g): keys a row of
    // 128 bytes after the other, with the 16-byte vectors of row r at place (v ^ (r >> 1) & 7), values as two halves
    // of 32 columns, 64 bytes a row. Wavefront w stages blocks of tokens 2 w and 2 w + 1. Those tokens lie in one page
    // each: page id and address are scalars, the lane's place in them never changes.
    const int last = max(w.q.n - 1, 0) & ~7, log2 = C.page_log2;
    const __attribute__((address_space(4))) int32_t* table =
        (const __attribute__((address_space(4))) int32_t*)(C.table + size_t(w.r) * C.width);
    const uint32_t pages = uint32_t(C.c.pages), page_rows = uint32_t(C.c.H) << log2;
    const uint8_t* const k0 = static_cast<const uint8_t*>(C.c.k) + (size_t(w.kvh) << log2) * kRowBytes;
    const uint8_t* const v0 = static_cast<const uint8_t*>(C.c.v) + (size_t(w.kvh) << log2) * kRowBytes;
    auto token_of = [&](int t, int j) { return uint32_t(min(t * kTile + 8 * NB * wave + 8 * j, last)); };
    const uint32_t first_seen = C.window ? uint32_t(max(past + t0 + 1 - C.window, 0)) : 0u;
    uint32_t ids[NB], bad = 0;
    auto load_ids = [&](int t) {
#pragma unroll
        for (int j = 0; j < NB; ++j) ids[j] = uint32_t(table[token_of(t, j) >> log2]);
    };
    uint32_t key_off[NB], value_off;         // bytes, in the tokens' rows
#pragma unroll
    for (int j = 0; j < NB; ++j)
        key_off[j] = (lane >> 3) * kRowBytes + (E ? 8 : 16) * ((lane & 7) ^ (((lane >> 4) & 3) | ((NB * wave + j) & 1) << 2));
    value_off = ((lane >> 2) & 7) * kRowBytes + (E ? 8 : 16) * (4 * h + (lane & 3));
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
                       uint32_t(uintptr_t((__attribute__((address_space(3))) uint8_t*)&stored[0][0][0]))) + 1024 * NB * wave;
    u32x2 kr[E ? NB * CB : 1], vr[E ? NB * CB : 1];
    float sr = 0.f;
    auto stage = [&](int t, int buf) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const uint32_t id = ids[j] < pages ? ids[j] : 0u;
            // (not 0 for an id outside the cache; the tokens before the block's first window may be in no page)
            bad |= token_of(t, j) + 8 > first_seen ? id ^ ids[j] : 0u;
            const uint64_t at = (uint64_t(id) * page_rows + (token_of(t, j) & ((1u << log2) - 1))) * kRowBytes;
            const uint8_t* k = k0 + at;
            const uint8_t* v = v0 + at;
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                if constexpr (E) {
                    kr[j * CB + c] = *reinterpret_cast<const u32x2*>(k + 64 * c + key_off[j]);
                    vr[j * CB + c] = *reinterpret_cast<const u32x2*>(v + 64 * c + value_off);
                } else {
                    const uint32_t to = lds0 + 2 * T::kTileBytes * buf + 1024 * (TB * c + j);
                    lds_load16_async(k + 128 * c, key_off[j], to);
                    lds_load16_async(v + 128 * c, value_off, to + T::kTileBytes);
                }
            }
        }
        if constexpr (E) {
            // scales of the tile's tokens: keys' by wavefront 0, values' by wavefront 1
            if (wave < 2 && lane < kTile) {
                const int tok = min(t * kTile + lane, max(w.q.n - 1, 0));
                uint32_t page = uint32_t(C.table[size_t(w.r) * C.width + (tok >> log2)]);
                page = page < pages ? page : 0;
                sr = (wave ? C.c.v_scale : C.c.k_scale)[uint64_t(page) * page_rows + (uint32_t(w.kvh) << log2) + (tok & ((1 << log2) - 1))];
            }
        }
    };
    auto put = [&](int buf) {                            // 8-bit rows, converted
        if constexpr (E) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int c = 0; c < CB; ++c) {
                    uint8_t* to = &stored[buf][0][1024 * (TB * c + NB * wave + j) + lane * 16];
                    *reinterpret_cast<u32x4*>(to) = e4m3_to8<T::ST>(kr[j * CB + c]);
                    *reinterpret_cast<u32x4*>(to + T::kTileBytes) = e4m3_to8<T::VT>(vr[j * CB + c]);
                }
            if (wave < 2 && lane < kTile) reinterpret_cast<float*>(&scales[buf][wave][0])[lane] = sr;
        }
    };

    // ------------------------------------------------------------------ one tile
    // Infinities and NaN among the values of a tile that some row does not see whole stay out of the products, where
    // a weight of 0 would make NaN of them: each wavefront looks through its tokens; where there are any, they
    // become 0 and their columns' bits are set. The rows that see such a token get their NaN behind the products.
    auto strange_values = [&](int t, int buf) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < NB * CB; ++i) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(&stored[buf][1][1024 * (TB * (i / NB) + NB * wave + i % NB) + lane * 16]);
            any |= not_finite<T::VT>(x[0]) | not_finite<T::VT>(x[1]) | not_finite<T::VT>(x[2]) | not_finite<T::VT>(x[3]);
        }
        if (__any(any != 0) && lane == 0) strange = t + 1;
        __syncthreads();
        if (strange != t + 1) return false;
#pragma unroll 1
        for (int i = 0; i < NB * CB; ++i) {
            u32x4* at = reinterpret_cast<u32x4*>(&stored[buf][1][1024 * (TB * (i / NB) + NB * wave + i % NB) + lane * 16]);
            u32x4 x = *at;
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t f = not_finite<T::VT>(x[e]) >> 15;          // bits 0 and 16
                bits |= ((f | f >> 15) & 3u) << (2 * e);
                x[e] &= ~(f * 0xFFFFu);
            }
            *at = x;
            // the lane holds columns 8 (lane % 4) ..+7 of half h of row (lane / 4) % 8
            reinterpret_cast<uint8_t*>(&strange_bits[8 * (NB * wave + i % NB) + ((lane >> 2) & 7)][2 * (i / NB) + h])[lane & 3] = uint8_t(bits);
        }
        __syncthreads();
        return true;
    };
    auto poison_rows = [&](int base) {
#pragma unroll
        for (int db = 0; db < DB; ++db) {
            uint32_t bits = 0;
            const int from = max(lower - base, 0), to = min(limit - base, kTile);
            for (int i = from; i < to; ++i) bits |= strange_bits[i][db];
            bits >>= 4 * h;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[db][i] = __uint_as_float(__float_as_uint(acc[db][i]) |
                                             (uint32_t(int(bits << (31 - 8 * (i >> 2) - (i & 3))) >> 31) & 0x7FC00000u));      // (NaN)
        }
    };

    // The lane's places: vector 2 i + h of token `col` (4 of them, then 64 columns further), and, for the transposing
    // reads, 4 columns of token 4 h + (l % 16) / 4 of 8
    uint32_t key_at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) key_at[i] = (col >> 3) * 1024 + (col & 7) * 128 + (((2 * i + h) ^ ((col >> 1) & 7)) << 4);
    const uint32_t value_at = (4 * h + ((lane & 15) >> 2)) * 64 + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;

    auto compute = [&](int t, int buf) {
        const bool partial = t < whole_from || t >= whole_to;
        const bool found = partial && strange_values(t, buf);
        if (t < any_from || t >= any_to) return;
        int to = limit - t * kTile - 4 * h, from = lower - t * kTile - 4 * h;         // of the lane's tokens
        f32x16 s[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            s[b] = f32x16{};
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(&stored[buf][0][key_at[i & 3] + 1024 * TB * (i >> 2) + 4096 * b]);
                s[b] = S::mul(a, qf[i], s[b]);
            }
            if constexpr (E) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 ks = scales[buf][0][8 * b + 2 * g + h];
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[b][4 * g + e] *= ks[e];
                }
            }
        }
        if (partial) {
            asm volatile("" : "+v"(to), "+v"(from));             // (or every tile would go through the selections)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][i] = hide(s[b][i], to - 1 - (32 * b + 8 * (i >> 2) + (i & 3)));
            if (windowed)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[b][i] = hide(s[b][i], 32 * b + 8 * (i >> 2) + (i & 3) - from);
        }
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
        top = max_xor32(top);
        if (__any((top - m) * mul > kThreshold)) {
            const float m_new = fmaxf(m, top);
            const float keep = m_new == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - m_new) * mul);
            weights() *= keep;
#pragma unroll
            for (int db = 0; db < DB; ++db) acc[db] *= keep;
            m = m_new;
        }
        float ref = (m == -INFINITY ? 0.f : m * mul) - T::kShift;
        if (__any(!(fabsf(ref) < 0x1p8f))) {
            // Scores far from 0: their differences first. (The reference is a rounded product, by which the exponents
            // are off, up to half of its last place: 2^-17 here, but 2^7 from 2^31 on.)
            const float by = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][i] -= by;
            ref = -T::kShift;
        }
        u32x4 p[2 * NB], p2[T::kTwoP ? 2 * NB : 1];
        float tile_l = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) e[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][4 * g + k], mul, -ref));
                tile_l += (e[0] + e[1]) + (e[2] + e[3]);
                if constexpr (E) {
                    const f32x4 vs = scales[buf][1][8 * b + 2 * g + h];
#pragma unroll
                    for (int k = 0; k < 4; ++k) e[k] *= vs[k];
                    if (partial) {                              // (a hidden token's scale may be anything)
                        asm volatile("" : "+v"(to), "+v"(from));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int tok = 32 * b + 8 * g + k;
                            e[k] = __uint_as_float(__float_as_uint(e[k]) & ~uint32_t(((to - 1 - tok) | (tok - from)) >> 31));
                        }
                    }
                }
                u32x4& x = p[2 * b + (g >> 1)];
                x[2 * (g & 1)] = pack2<T::VT>(e[0], e[1]);
                x[2 * (g & 1) + 1] = pack2<T::VT>(e[2], e[3]);
                if constexpr (T::kTwoP) {
                    u32x4& y = p2[2 * b + (g >> 1)];
                    const uint32_t h0 = x[2 * (g & 1)], h1 = x[2 * (g & 1) + 1];
                    y[2 * (g & 1)] = pack2<T::VT>(e[0] - low<T::VT>(h0), e[1] - high<T::VT>(h0));
                    y[2 * (g & 1) + 1] = pack2<T::VT>(e[2] - low<T::VT>(h1), e[3] - high<T::VT>(h1));
                }
            }
        {
            // The sum and what its rounding leaves (TwoSum: Knuth, The Art of Computer Programming 2, 4.2.2): one rounding
            // after the other would take 9e-4 off a row of 131072 equal weights, all on one side
            const f32x2 l = weights();
            const float sum = l[0] + tile_l, added = sum - l[0];
            weights() = f32x2{sum, l[1] + ((l[0] - (sum - added)) + (tile_l - added))};
        }
        const uint8_t* values = &stored[buf][1][value_at];
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int s4 = 0; s4 < 2 * NB; ++s4) {         // 16 tokens
                u32x4 a;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const u32x2 x = __builtin_bit_cast(u32x2, read_transposed(values + 1024 * (TB * (db >> 1) + 2 * s4 + u) + 512 * (db & 1)));
                    a[2 * u] = x[0];
                    a[2 * u + 1] = x[1];
                }
                acc[db] = V::mul(a, p[s4], acc[db]);
                if constexpr (T::kTwoP) acc[db] = V::mul(a, p2[s4], acc[db]);
            }
        if (found) poison_rows(t * kTile);
    };

    // ------------------------------------------------------------------ the part's tiles
    if (tiles.from < tiles.to) {
        load_ids(tiles.from);
        stage(tiles.from, 0);
        load_ids(min(tiles.from + 1, tiles.to - 1));
        put(0);
    }
    int buf = 0;
    for (int t = tiles.from; t < tiles.to; ++t) {
        lds_loads_wait();
        __syncthreads();
        if (t + 1 < tiles.to) {
            stage(t + 1, buf ^ 1);
            load_ids(min(t + 2, tiles.to - 1));
        }
        compute(t, buf);
        if (E && t + 1 < tiles.to) put(buf ^ 1);
        buf ^= 1;
    }
    __syncthreads();
    if (bad && lane == 0) bad_page = 1;
    __syncthreads();

    // ------------------------------------------------------------------ sums out
    const auto& B = arguments_again();
    float l = w.q.bad || bad_page ? __builtin_nanf("") : add_xor32_f32(weights()[0] + weights()[1]);
    const int j = wave * 32 + col, token = j / B.heads, head = j - token * B.heads;
    if (token >= tokens || head >= min(B.heads, B.G - w.hb * B.heads)) return;
    if (B.scale == 0.f) {                                    // (0 times an infinity or a NaN is a NaN)
        const uint16_t* q = static_cast<const uint16_t*>(B.q) + (int64_t(w.q.first) + t0 + token) * B.q_row +
                            int64_t(w.kvh * B.G + w.hb * B.heads + head) * B.q_head + 8 * h;
        uint32_t any = 0;
        for (int i = 0; i < KS; ++i) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(q + 16 * i);
            any |= not_finite<QT>(x[0]) | not_finite<QT>(x[1]) | not_finite<QT>(x[2]) | not_finite<QT>(x[3]);
        }
        if (any | __shfl_xor(any, 32)) l = __builtin_nanf("");
    }
    if (w.parts == 1) {
        const size_t row = (size_t(w.q.first) + t0 + token) * B.Hq + w.kvh * B.G + w.hb * B.heads + head;
        const float by = l == 0.f ? 0.f : 1.f / l;
        uint16_t* o = static_cast<uint16_t*>(B.o) + row * D + 4 * h;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<u32x2*>(o + 32 * db + 8 * g) =
                    scaled<QT>(f32x4{acc[db][4 * g], acc[db][4 * g + 1], acc[db][4 * g + 2], acc[db][4 * g + 3]}, by);
        if (B.lse && h == 0)
            B.lse[row] = l == 0.f ? -INFINITY : m * (B.scale == 0.f ? 1.f : fabsf(B.scale)) + logf(l * (1.f / (1 << T::kShift)));
    } else {
        const size_t at = size_t(w.slot) * kRows + j;
        float* o = B.part_o + at * D + 4 * h;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4*>(o + 32 * db + 8 * g) =
                    f32x4{acc[db][4 * g], acc[db][4 * g + 1], acc[db][4 * g + 2], acc[db][4 * g + 3]};
        if (h == 0) {
            B.part_ml[2 * at] = m;
            B.part_ml[2 * at + 1] = l;
        }
    }
}

// Joins the parts of split blocks: as many workgroups as parts, the p-th of a block for the
// p-th share of its rows, a lane per 4 columns, with the sums of 8 parts on their way at a time (16 new
// tokens of 16000, 128 parts: 34 us a call; 59 with one part after the other).
constexpr int kOnWay = 8;
template <int QT, int D, int SHIFT>
__global__ void __launch_bounds__(kThreads) join_chunks_kernel(const ChunkArgs A) {
    Work w;
    if (!find_work<true>(A, blockIdx.x, w)) return;
    const int rows = min(A.tokens, w.q.m - w.block * A.tokens) * A.heads;
    const int r0 = int(int64_t(rows) * w.part / w.parts), r1 = int(int64_t(rows) * (w.part + 1) / w.parts);
    const int heads_here = min(A.heads, A.G - w.hb * A.heads);
    const int64_t step = int64_t(A.c.H) * A.head_blocks;          // slots between a block's parts
    const Tiles all = tiles_of(A, w.q, w.block, 0, 1);
    const int64_t n = all.to - all.from;
    const float natural = A.scale == 0.f ? 1.f : fabsf(A.scale), mul = natural * kLog2e;
    for (int e = threadIdx.x; e < (r1 - r0) * (D / 4); e += kThreads) {
        const int j = r0 + e / (D / 4), d = 4 * (e % (D / 4));
        const int token = j / A.heads, head = j - token * A.heads;
        if (head >= heads_here) continue;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, l = 0.f;
        for (int p0 = 0; p0 < w.parts; p0 += kOnWay) {
            float mc[kOnWay], lc[kOnWay];
            f32x4 vc[kOnWay];
            bool some[kOnWay];
            float top = m;
#pragma unroll
            for (int i = 0; i < kOnWay; ++i) {
                const int p = p0 + i;
                const int64_t slot = w.slot0 + p * step;
                // (a part without tiles has stored nothing; slot 0 is read in its place, and left out)
                some[i] = p < w.parts && (n >= w.parts || n * p / w.parts < n * (p + 1) / w.parts) && uint64_t(slot) < uint64_t(A.slots);
                const size_t at = size_t(some[i] ? slot : 0) * kRows + j;
                mc[i] = A.part_ml[2 * at];
                lc[i] = A.part_ml[2 * at + 1];
                vc[i] = *reinterpret_cast<const f32x4*>(A.part_o + at * D + d);
            }
#pragma unroll
            for (int i = 0; i < kOnWay; ++i) {
                mc[i] = some[i] ? mc[i] : -INFINITY;
                top = fmaxf(top, mc[i]);
            }
            const float ref = top == -INFINITY ? 0.f : top, f = __builtin_amdgcn_exp2f((m - ref) * mul);
            l *= f;
            v *= f;
            m = top;
#pragma unroll
            for (int i = 0; i < kOnWay; ++i)
                if (some[i]) {
                    const float fc = __builtin_amdgcn_exp2f((mc[i] - ref) * mul);
                    l += lc[i] * fc;
                    v += vc[i] * fc;
                }
        }
        const size_t row = (size_t(w.q.first) + w.block * A.tokens + token) * A.Hq + w.kvh * A.G + w.hb * A.heads + head;
        const float by = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(A.o) + row * D + d) = scaled<QT>(v, by);
        if (A.lse && d == 0) A.lse[row] = l == 0.f ? -INFINITY : m * natural + logf(l * (1.f / (1 << SHIFT)));
    }
}

template <int KV, int QT, int D, int LIMBS>
hipError_t chunk_d(ChunkArgs a, hipStream_t s) {
    constexpr int64_t most = kLaunchItems / kThreads;
    for (; a.launched < a.groups; a.launched += most) {
        const int64_t groups = a.groups - a.launched < most ? a.groups - a.launched : most;
        chunk_kernel<KV, QT, D, LIMBS><<<unsigned(groups), kThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.slots) return hipSuccess;
    join_chunks_kernel<QT, D, Chunk<KV, QT, D, LIMBS>::kShift><<<unsigned(a.slots), kThreads, 0, s>>>(a);
    return hipGetLastError();
}
template <int KV, int QT, int LIMBS>
hipError_t chunk_l(const ChunkArgs& a, hipStream_t s) {
    switch (a.c.D) {
        case 64: return chunk_d<KV, QT, 64, LIMBS>(a, s);
        case 128: return chunk_d<KV, QT, 128, LIMBS>(a, s);
        default: return chunk_d<KV, QT, 256, LIMBS>(a, s);
    }
}
template <int KV, int QT>
hipError_t chunk_t(const ChunkArgs& a, hipStream_t s) {
    if constexpr (KV == WB_E4M3 && QT == WB_F16) return chunk_l<KV, QT, 2>(a, s);
    else return a.limbs == 1 ? chunk_l<KV, QT, 1>(a, s) : chunk_l<KV, QT, 2>(a, s);
}

}  // namespace

// Tokens of a part at least, where a request's block is split. All tiles are cut into about as many parts as the device
// holds workgroups (512): twice as many make 64 requests of drafts 106 us, not 97 (the starts of parts, their sums and
// the join), and windows 73, not 59. (One request's 16 new tokens of 1000: 14.4 us with parts of 128 tokens, 19.0 with 256;
// of 4000 18.4 and 18.7.)
constexpr int kPartTokens = 128;

ChunkPlan chunk_plan(const wb_kv_cache& c, int N, int R, int Hq, int width) {
    const int G = Hq / c.H;
    ChunkPlan p;
    p.heads = G < kRows ? G : kRows;
    p.head_blocks = (G + p.heads - 1) / p.heads;
    p.tokens = kRows / p.heads;
    p.tile_log2 = tile_log2(c.D);
    p.part_tiles = kPartTokens >> p.tile_log2;
    p.target = 256 * kWavesPerSimd;
    const int64_t by_tokens = int64_t(N) / p.tokens + R, blocks = (N < by_tokens ? N : by_tokens) * int64_t(c.H) * p.head_blocks;
    const int64_t tiles = (int64_t(width) * c.page + (1 << p.tile_log2) - 1) >> p.tile_log2;
    p.slots = 0;
    if (tiles > p.part_tiles) {
        // (a block of s tiles has ceil(s / t) parts of at most t >= all tiles / target: fewer than
        // 2 s / t where that is more than one)
        const int64_t most = blocks * ((tiles + p.part_tiles - 1) / p.part_tiles);
        p.slots = most < 2 * p.target ? most : 2 * p.target;
    }
    p.groups = blocks + (p.slots ? p.target : 0);
    p.part_o_bytes = size_t(p.slots) * kRows * c.D * 4;
    p.part_ml_bytes = size_t(p.slots) * kRows * 8;
    p.before_bytes = R > 64 ? size_t(R + 2) * 8 : 0;
    return p;
}

hipError_t launch_chunk(const ChunkArgs& a, hipStream_t s) {
    if (a.before) {
        count_requests_kernel<<<1, kCountThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.c.dtype == WB_BF16) return chunk_t<WB_BF16, WB_BF16>(a, s);
    if (a.c.dtype == WB_F16) return chunk_t<WB_F16, WB_F16>(a, s);
    return a.q_dtype == WB_BF16 ? chunk_t<WB_E4M3, WB_BF16>(a, s) : chunk_t<WB_E4M3, WB_F16>(a, s);
}

}  // namespace wb
