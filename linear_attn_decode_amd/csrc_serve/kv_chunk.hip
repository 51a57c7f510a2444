// Attention of chunks of new tokens over a paged key-value cache (wbserve.h).
//
//   o_i = sum_t e^{s_it - m} v_t / sum_t e^{s_it - m},  s_it = scale q_i . k_t,  t <= position of i
//
// in one pass over the stored tokens with a running maximum.
#include "serve_device.hpp"

namespace wb {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4, kThreads = 64 * kWaves, kTile = 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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
    q.span = (q.n + kTile - 1) / kTile;
    if (A.window) q.span = min(q.span, int((int64_t(A.window) + A.tokens + 2 * kTile - 3) / kTile));
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

// The work of number `at`, among all parts, or among those of split blocks only. False: there
// are not so many. Every wavefront finds it for itself: lane l sums over requests [l per,
// (l + 1) per), a scan finds the lane, a second one the request among its.
template <bool SPLIT_ONLY>
__device__ __forceinline__ bool find_work(const ChunkArgs& A, int64_t at, Work& w) {
    const int lane = threadIdx.x & 63, per = (A.R + 63) / 64;
    const int per_block = A.c.H * A.head_blocks;
    int64_t cost = 0;
    for (int i = 0; i < per; ++i) {
        const int r = lane * per + i;
        if (r < A.R) {
            const Request q = request_of(A, r);
            cost += int64_t(q.blocks) * q.span;
        }
    }
    cost = lane64(wave_scan(cost), 63) * per_block;
    const int64_t most64 = max(int64_t(A.part_tiles), quotient64(cost + A.target - 1, int64_t(A.target)));
    const int most = int(min(most64, int64_t(1) << 30));         // tiles of a part
    auto parts_in = [&](const Request& q) { return (q.span + most - 1) / most; };
    // (parts in the lower half, those of split blocks in the upper one)
    auto count = [&](const Request& q) {
        const int parts = parts_in(q);
        const int64_t n = int64_t(q.blocks) * per_block * parts;
        return n | (parts > 1 ? n : 0) << 32;
    };
    auto key = [&](int64_t v) { return SPLIT_ONLY ? v >> 32 : v & 0xFFFFFFFF; };
    int64_t mine = 0;
    for (int i = 0; i < per; ++i)
        if (lane * per + i < A.R) mine += count(request_of(A, lane * per + i));
    const int64_t upto = wave_scan(mine);
    if (key(lane64(upto, 63)) <= at) return false;
    const int who = __ffsll((unsigned long long)__ballot(key(upto) > at)) - 1;
    int64_t before = lane64(upto, who) - lane64(mine, who);
    w.r = min((who + 1) * per, A.R) - 1;
    for (int base = who * per; per > 1 && base < (who + 1) * per; base += 64) {
        const int r = base + lane;
        const int64_t n = r < (who + 1) * per && r < A.R ? count(request_of(A, r)) : 0;
        const int64_t sum = before + wave_scan(n);
        const uint64_t past = __ballot(key(sum) > at);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            w.r = base + l;
            before = lane64(sum, l) - lane64(n, l);
            break;
        }
        before = lane64(sum, 63);
    }
    w.r = __builtin_amdgcn_readfirstlane(w.r);
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

// Key tiles [from, to) of a part
struct Tiles {
    int from, to;
};
__device__ __forceinline__ Tiles tiles_of(const ChunkArgs& A, const Request& q, int block, int part, int parts) {
    const int t0 = block * A.tokens, t1 = min(t0 + A.tokens, q.m);       // new tokens of the block
    const int past = q.n - q.m;
    const int lo = A.window ? max(past + t0 - A.window + 1, 0) / kTile : 0, hi = q.bad ? 0 : (past + t1 + kTile - 1) / kTile;
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

// 16 bytes a lane from `base` + `off` bytes straight to LDS (the lane's after `to`, which like `base` is the same for
// all lanes). Written as assembly because behind the builtin the compiler lets every later read of LDS wait for all
// such loads: the next tile's would not stay in flight behind this one's products. It writes no register, so there is
// none for the compiler to use too early; lds_loads_wait() and a barrier come before the data is read.
__device__ __forceinline__ void lds_load16_async(const void* base, uint32_t off, const uint8_t* to) {
    const uint32_t at = uint32_t(uintptr_t((const __attribute__((address_space(3))) uint8_t*)to));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(at)), "v"(off), "s"(base)
                 : "memory");
}

// 4 columns of a finished row out to o; the row's log-sum-exp with its first
template <int QT>
__device__ __forceinline__ u32x2 scaled(f32x4 v, float by) {
    return u32x2{pack2<QT>(v[0] * by, v[1] * by), pack2<QT>(v[2] * by, v[3] * by)};
}

constexpr int waves_per_simd(int D, int NQ) { return D <= 128 && NQ == 1 ? 2 : 1; }

// KV: the cache's type; QT: the type of q and o; D: columns; NQ: blocks of 32 rows a wavefront
template <int KV, int QT, int D, int NQ>
struct Chunk {
    static constexpr int ST = QT;                                    // operands of the scores
    static constexpr int VT = KV == WB_E4M3 ? WB_BF16 : KV;          // of the values
    static constexpr bool kTwoP = KV == WB_E4M3 && QT == WB_F16;
    static constexpr int KS = D / 16;                                // score products of 32 tokens
    static constexpr int DB = D / 32;                                // blocks of value columns
    static constexpr int CB = D / 64;                                // blocks of 64 columns
    static constexpr int kShift = VT == WB_F16 ? 11 : 0;             // weights enter as 2^kShift times their value
    static constexpr int kRows = 32 * NQ * kWaves;
    static constexpr int kTileBytes = kTile * D * 2;
};

template <int KV, int QT, int D, int NQ>
__global__ void __launch_bounds__(kThreads, waves_per_simd(D, NQ)) chunk_kernel(const ChunkArgs A) {
    using T = Chunk<KV, QT, D, NQ>;
    using S = Mat32<T::ST>;
    using V = Mat32<T::VT>;
    constexpr int KS = T::KS, DB = T::DB, CB = T::CB;
    constexpr bool E = KV == WB_E4M3;
    constexpr float kThreshold = 4.f;
    __shared__ __attribute__((aligned(1024))) uint8_t stored[2][2][T::kTileBytes];        // [buffer][keys, values]
    __shared__ f32x4 scales[2][2][kTile / 4];
    __shared__ uint32_t strange_bits[kTile][DB];                     // of the tile's values: columns of each token
    __shared__ int strange, bad_page;

    Work w;
    if (!find_work<false>(A, blockIdx.x, w)) return;
    const Tiles tiles = tiles_of(A, w.q, w.block, w.part, w.parts);
    if (w.parts > 1 && (tiles.from >= tiles.to || uint64_t(w.slot) >= uint64_t(A.slots))) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, col = lane & 31;
    if (tid == 0) strange = bad_page = 0;

    // The lane's rows of q: row j of the block is head j % heads of token j / heads
    const int heads = A.heads, heads_here = min(heads, A.G - w.hb * heads);
    const int past = w.q.n - w.q.m, t0 = w.block * A.tokens, tokens = min(A.tokens, w.q.m - t0);
    int64_t row_at[NQ];                 // row of o and lse, or -1
    int limit[NQ], lower[NQ];           // tokens [lower, limit) are seen
    u32x4 qf[NQ][KS];
#pragma unroll
    for (int qn = 0; qn < NQ; ++qn) {
        const int j = (wave * NQ + qn) * 32 + col, token = j / heads, head = j - token * heads;
        const bool ok = token < tokens && head < heads_here;
        const int64_t row = int64_t(w.q.first) + t0 + token;
        const int hq = w.kvh * A.G + w.hb * heads + head;
        row_at[qn] = ok ? row * A.Hq + hq : -1;
        limit[qn] = ok ? past + t0 + token + 1 : 0;
        lower[qn] = A.window ? max(limit[qn] - A.window, 0) : 0;
        const uint16_t* q = static_cast<const uint16_t*>(A.q) + row * A.q_row + int64_t(hq) * A.q_head + 8 * h;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            qf[qn][i] = u32x4{0, 0, 0, 0};
            if (ok && A.scale != 0.f) qf[qn][i] = *reinterpret_cast<const u32x4*>(q + 16 * i);
            if (A.scale < 0.f) qf[qn][i] ^= 0x80008000u;
        }
    }
    // (a scale of 0: scores of 0)
    const float natural = A.scale == 0.f ? 1.f : fabsf(A.scale), mul = natural * kLog2e;
    // of the wavefront: the tokens that any row sees, and those that all of its rows see
    const int row0 = wave * NQ * 32;
    const int first_token = row0 / heads, last_token = min((row0 + NQ * 32 - 1) / heads, tokens - 1);
    const bool active = first_token < tokens;
    const int any_hi = past + t0 + last_token + 1, all_hi = past + t0 + first_token + 1;
    const int any_lo = A.window ? max(all_hi - A.window, 0) : 0, all_lo = A.window ? max(any_hi - A.window, 0) : 0;

    f32x16 acc[NQ][DB];
    float m[NQ], l[NQ];
#pragma unroll
    for (int qn = 0; qn < NQ; ++qn) {
#pragma unroll
        for (int i = 0; i < DB; ++i) acc[qn][i] = f32x16{};
        m[qn] = -INFINITY;
        l[qn] = 0.f;
    }

    // ------------------------------------------------------------------ staging
    // A tile lies in LDS as blocks of 8 tokens by 64 columns, 1 KB each, block (c, g) at 1024 (8 c + g): keys a row of
    // 128 bytes after the other, with the 16-byte vectors of row r at place (v ^ (r >> 1) & 7), values as two halves
    // of 32 columns, 64 bytes a row. Wavefront w stages blocks of tokens 2 w and 2 w + 1. Those tokens lie in one page
    // each: page id and address are scalars, the lane's place in them never changes.
    const int last = max(w.q.n - 1, 0) & ~7;
    const __attribute__((address_space(4))) int32_t* table =
        (const __attribute__((address_space(4))) int32_t*)(A.table + size_t(w.r) * A.width);
    const int page_mask = (1 << A.page_log2) - 1;
    auto token_of = [&](int t, int j) { return min(t * kTile + 16 * wave + 8 * j, last); };
    int ids[2];
    auto load_ids = [&](int t) {
#pragma unroll
        for (int j = 0; j < 2; ++j) ids[j] = table[uint32_t(token_of(t, j)) >> A.page_log2];
    };
    int bad = 0;
    const uint32_t pages = uint32_t(A.c.pages);
    auto base_of = [&](int t, int j) -> size_t {          // first value of the tokens
        const bool ok = uint32_t(ids[j]) < pages;
        bad |= !ok;
        const uint64_t row = (uint64_t(ok ? uint32_t(ids[j]) : 0u) * uint32_t(A.c.H) + uint32_t(w.kvh)) << A.page_log2;
        return (row + uint32_t(token_of(t, j) & page_mask)) * D;
    };
    uint32_t key_off[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) key_off[j] = uint32_t((lane >> 3) * D + 8 * ((lane & 7) ^ (((lane >> 4) & 3) | j << 2)));
    const uint32_t value_off = uint32_t(((lane >> 2) & 7) * D + 32 * h + 8 * (lane & 3));
    u32x2 kr[E ? 2 * CB : 1], vr[E ? 2 * CB : 1];
    float sr = 0.f;
    auto stage = [&](int t, int buf) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const size_t base = base_of(t, j);
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                if constexpr (E) {
                    kr[j * CB + c] = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(A.c.k) + base + 64 * c + key_off[j]);
                    vr[j * CB + c] = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(A.c.v) + base + 64 * c + value_off);
                } else {
                    uint8_t* to = &stored[buf][0][1024 * (8 * c + 2 * wave + j)];
                    lds_load16_async(static_cast<const uint16_t*>(A.c.k) + base + 64 * c, 2 * key_off[j], to);
                    lds_load16_async(static_cast<const uint16_t*>(A.c.v) + base + 64 * c, 2 * value_off, to + T::kTileBytes);
                }
            }
        }
        if constexpr (E) {
            // scales of the tile's tokens: keys' by wavefront 0, values' by wavefront 1
            if (wave < 2) {
                const int tok = min(t * kTile + lane, max(w.q.n - 1, 0));
                int page = A.table[size_t(w.r) * A.width + (tok >> A.page_log2)];
                page = page >= 0 && page < A.c.pages ? page : 0;
                sr = (wave ? A.c.v_scale : A.c.k_scale)[((size_t(page) * A.c.H + w.kvh) << A.page_log2) + (tok & page_mask)];
            }
        }
    };
    auto put = [&](int buf) {                            // 8-bit rows, converted
        if constexpr (E) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < CB; ++c) {
                    uint8_t* to = &stored[buf][0][1024 * (8 * c + 2 * wave + j) + lane * 16];
                    *reinterpret_cast<u32x4*>(to) = e4m3_to8<T::ST>(kr[j * CB + c]);
                    *reinterpret_cast<u32x4*>(to + T::kTileBytes) = e4m3_to8<T::VT>(vr[j * CB + c]);
                }
            if (wave < 2) reinterpret_cast<float*>(&scales[buf][wave][0])[lane] = sr;
        }
    };

    // ------------------------------------------------------------------ one tile
    // The lane's places: vector 2 i + h of token `col` (4 of them, then 64 columns further), and, for the transposing
    // reads, 4 columns of token 4 h + (l % 16) / 4 of 8
    uint32_t key_at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) key_at[i] = (col >> 3) * 1024 + (col & 7) * 128 + (((2 * i + h) ^ ((col >> 1) & 7)) << 4);
    const uint32_t value_at = (4 * h + ((lane & 15) >> 2)) * 64 + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;

    // Infinities and NaN among the values of a tile that some row does not see whole stay out of the products, where
    // a weight of 0 would make NaN of them: each wavefront looks through its tokens; where there are any, they
    // become 0 and their columns' bits are set. The rows that see such a token get their NaN behind the products.
    auto strange_values = [&](int t, int buf) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 2 * CB; ++i) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(&stored[buf][1][1024 * (8 * (i >> 1) + 2 * wave + (i & 1)) + lane * 16]);
            any |= not_finite<T::VT>(x[0]) | not_finite<T::VT>(x[1]) | not_finite<T::VT>(x[2]) | not_finite<T::VT>(x[3]);
        }
        if (__any(any != 0) && lane == 0) strange = t + 1;
        __syncthreads();
        if (strange != t + 1) return false;
#pragma unroll 1
        for (int i = 0; i < 2 * CB; ++i) {
            u32x4* at = reinterpret_cast<u32x4*>(&stored[buf][1][1024 * (8 * (i >> 1) + 2 * wave + (i & 1)) + lane * 16]);
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
            reinterpret_cast<uint8_t*>(&strange_bits[16 * wave + 8 * (i & 1) + ((lane >> 2) & 7)][2 * (i >> 1) + h])[lane & 3] = uint8_t(bits);
        }
        __syncthreads();
        return true;
    };
    auto poison_rows = [&](int base) {
#pragma unroll
        for (int qn = 0; qn < NQ; ++qn)
#pragma unroll
            for (int db = 0; db < DB; ++db) {
                uint32_t bits = 0;
                const int from = max(lower[qn] - base, 0), to = min(limit[qn] - base, kTile);
                for (int i = from; i < to; ++i) bits |= strange_bits[i][db];
                bits >>= 4 * h;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (bits >> (8 * (i >> 2) + (i & 3)) & 1) acc[qn][db][i] = __builtin_nanf("");
            }
    };
    auto values = [&](int buf, const u32x4 (&p)[NQ][4], const u32x4 (&p2)[T::kTwoP ? NQ : 1][4]) {
        const uint8_t* from = &stored[buf][1][value_at];
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int s = 0; s < 4; ++s) {                 // 16 tokens
                u32x4 a;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const u32x2 x = __builtin_bit_cast(u32x2, read_transposed(from + 1024 * (8 * (db >> 1) + 2 * s + u) + 512 * (db & 1)));
                    a[2 * u] = x[0];
                    a[2 * u + 1] = x[1];
                }
#pragma unroll
                for (int qn = 0; qn < NQ; ++qn) {
                    acc[qn][db] = V::mul(a, p[qn][s], acc[qn][db]);
                    if constexpr (T::kTwoP) acc[qn][db] = V::mul(a, p2[qn][s], acc[qn][db]);
                }
            }
    };

    auto compute = [&](int t, int buf, bool found) {
        const int base = t * kTile;
        if (!active || base >= any_hi || base + kTile <= any_lo) return;
        const bool masked = base + kTile > all_hi || base < all_lo;
        f32x16 s[NQ][2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int qn = 0; qn < NQ; ++qn) s[qn][b] = f32x16{};
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(&stored[buf][0][key_at[i & 3] + 8192 * (i >> 2) + 4096 * b]);
#pragma unroll
                for (int qn = 0; qn < NQ; ++qn) s[qn][b] = S::mul(a, qf[qn][i], s[qn][b]);
            }
            if constexpr (E) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 ks = scales[buf][0][8 * b + 2 * g + h];
#pragma unroll
                    for (int qn = 0; qn < NQ; ++qn)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[qn][b][4 * g + e] *= ks[e];
                }
            }
        }
        if (masked) {
#pragma unroll
            for (int qn = 0; qn < NQ; ++qn) {
                const int to = limit[qn] - base - 4 * h, from = lower[qn] - base - 4 * h;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (32 * b + 8 * (i >> 2) + (i & 3) >= to) s[qn][b][i] = -INFINITY;
                if (A.window)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (32 * b + 8 * (i >> 2) + (i & 3) < from) s[qn][b][i] = -INFINITY;
            }
        }
        u32x4 p[NQ][4], p2[T::kTwoP ? NQ : 1][4];
#pragma unroll
        for (int qn = 0; qn < NQ; ++qn) {
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[qn][b][i]);
            top = max_xor32(top);
            if (__any((top - m[qn]) * mul > kThreshold)) {
                const float m_new = fmaxf(m[qn], top);
                const float keep = m_new == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m[qn] - m_new) * mul);
                l[qn] *= keep;
#pragma unroll
                for (int db = 0; db < DB; ++db) acc[qn][db] *= keep;
                m[qn] = m_new;
            }
            float ref = (m[qn] == -INFINITY ? 0.f : m[qn] * mul) - T::kShift;
            if (__any(!(fabsf(ref) < 0x1p100f))) {
                // (scores near the ends of float32's range: their differences first)
                const float by = m[qn] == -INFINITY ? 0.f : m[qn];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[qn][b][i] -= by;
                ref = -T::kShift;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        e[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[qn][b][4 * g + k], mul, -ref));
                        l[qn] += e[k];
                    }
                    if constexpr (E) {
                        const f32x4 vs = scales[buf][1][8 * b + 2 * g + h];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            e[k] *= vs[k];
                            const int tok = base + 32 * b + 8 * g + 4 * h + k;
                            if (masked && (tok < lower[qn] || tok >= limit[qn])) e[k] = 0.f;      // (its scale may be anything)
                        }
                    }
                    u32x4& to = p[qn][2 * b + (g >> 1)];
                    to[2 * (g & 1)] = pack2<T::VT>(e[0], e[1]);
                    to[2 * (g & 1) + 1] = pack2<T::VT>(e[2], e[3]);
                    if constexpr (T::kTwoP) {
                        u32x4& to2 = p2[qn][2 * b + (g >> 1)];
                        const uint32_t h0 = to[2 * (g & 1)], h1 = to[2 * (g & 1) + 1];
                        to2[2 * (g & 1)] = pack2<T::VT>(e[0] - low<T::VT>(h0), e[1] - high<T::VT>(h0));
                        to2[2 * (g & 1) + 1] = pack2<T::VT>(e[2] - low<T::VT>(h1), e[3] - high<T::VT>(h1));
                    }
                }
        }
        values(buf, p, p2);
        if (found) poison_rows(base);
    };

    // ------------------------------------------------------------------ the part's tiles
    if (tiles.from < tiles.to) {
        load_ids(tiles.from);
        stage(tiles.from, 0);
        load_ids(min(tiles.from + 1, tiles.to - 1));
        put(0);
    }
    for (int t = tiles.from; t < tiles.to; ++t) {
        const int buf = (t - tiles.from) & 1;
        lds_loads_wait();
        __syncthreads();
        if (t + 1 < tiles.to) {
            stage(t + 1, buf ^ 1);
            load_ids(min(t + 2, tiles.to - 1));
        }
        const bool partial = (t + 1) * kTile > past + t0 + 1 || (A.window && t * kTile < past + t0 + tokens - A.window);
        const bool found = partial && strange_values(t, buf);
        compute(t, buf, found);
        if (E && t + 1 < tiles.to) put(buf ^ 1);
    }
    __syncthreads();
    if (bad && lane == 0) bad_page = 1;
    __syncthreads();
    const bool poison = w.q.bad || bad_page;

    // ------------------------------------------------------------------ sums out
#pragma unroll
    for (int qn = 0; qn < NQ; ++qn) {
        float total = add_xor32_f32(l[qn]);
        if (poison) total = __builtin_nanf("");
        if (w.parts == 1) {
            if (row_at[qn] < 0) continue;
            const float by = total == 0.f ? 0.f : 1.f / total;
            uint16_t* o = static_cast<uint16_t*>(A.o) + row_at[qn] * D;
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 v = {acc[qn][db][4 * g], acc[qn][db][4 * g + 1], acc[qn][db][4 * g + 2], acc[qn][db][4 * g + 3]};
                    *reinterpret_cast<u32x2*>(o + 32 * db + 8 * g + 4 * h) = scaled<QT>(v, by);
                }
            if (A.lse && h == 0)
                A.lse[row_at[qn]] = total == 0.f ? -INFINITY : m[qn] * natural + (logf(total) - T::kShift * kLn2);
        } else if (row_at[qn] >= 0) {
            const size_t at = size_t(w.slot) * T::kRows + (wave * NQ + qn) * 32 + col;
            float* o = A.part_o + at * D;
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<f32x4*>(o + 32 * db + 8 * g + 4 * h) =
                        f32x4{acc[qn][db][4 * g], acc[qn][db][4 * g + 1], acc[qn][db][4 * g + 2], acc[qn][db][4 * g + 3]};
            if (h == 0) {
                A.part_ml[2 * at] = m[qn];
                A.part_ml[2 * at + 1] = total;
            }
        }
    }
}

// Joins the parts of split blocks: as many workgroups as parts, the p-th of a block for the
// p-th share of its rows, a lane per 4 columns.
template <int QT, int D, int SHIFT>
__global__ void __launch_bounds__(kThreads) join_chunks_kernel(const ChunkArgs A) {
    Work w;
    if (!find_work<true>(A, blockIdx.x, w)) return;
    const int rows = min(A.tokens, w.q.m - w.block * A.tokens) * A.heads;
    const int r0 = int(int64_t(rows) * w.part / w.parts), r1 = int(int64_t(rows) * (w.part + 1) / w.parts);
    const int heads_here = min(A.heads, A.G - w.hb * A.heads);
    const int64_t step = int64_t(A.c.H) * A.head_blocks;          // slots between a block's parts
    const Tiles all = tiles_of(A, w.q, w.block, 0, 1);
    const float natural = A.scale == 0.f ? 1.f : fabsf(A.scale), mul = natural * kLog2e;
    for (int e = threadIdx.x; e < (r1 - r0) * (D / 4); e += kThreads) {
        const int j = r0 + e / (D / 4), d = 4 * (e % (D / 4));
        const int token = j / A.heads, head = j - token * A.heads;
        if (head >= heads_here) continue;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, l = 0.f;
        for (int p = 0; p < w.parts; ++p) {
            const int64_t slot = w.slot0 + p * step;
            const int64_t n = all.to - all.from;
            if (n * p / w.parts >= n * (p + 1) / w.parts || uint64_t(slot) >= uint64_t(A.slots)) continue;      // (a part without tiles)
            const size_t at = size_t(slot) * A.rows + j;
            const float mc = A.part_ml[2 * at], lc = A.part_ml[2 * at + 1];
            const f32x4 vc = *reinterpret_cast<const f32x4*>(A.part_o + at * D + d);
            const float top = fmaxf(m, mc), ref = top == -INFINITY ? 0.f : top;
            const float f = __builtin_amdgcn_exp2f((m - ref) * mul), fc = __builtin_amdgcn_exp2f((mc - ref) * mul);
            l = l * f + lc * fc;
            v = v * f + vc * fc;
            m = top;
        }
        const size_t row = (size_t(w.q.first) + w.block * A.tokens + token) * A.Hq + w.kvh * A.G + w.hb * A.heads + head;
        const float by = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(A.o) + row * D + d) = scaled<QT>(v, by);
        if (A.lse && d == 0) A.lse[row] = l == 0.f ? -INFINITY : m * natural + (logf(l) - SHIFT * kLn2);
    }
}

template <int KV, int QT, int D>
hipError_t chunk_d(const ChunkArgs& a, hipStream_t s) {
    if (D <= 128 && a.rows == 256) {
        if constexpr (D <= 128) chunk_kernel<KV, QT, D, 2><<<a.groups, kThreads, 0, s>>>(a);
    } else {
        chunk_kernel<KV, QT, D, 1><<<a.groups, kThreads, 0, s>>>(a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.slots) return e;
    join_chunks_kernel<QT, D, Chunk<KV, QT, D, 1>::kShift><<<unsigned(a.slots), kThreads, 0, s>>>(a);
    return hipGetLastError();
}
template <int KV, int QT>
hipError_t chunk_t(const ChunkArgs& a, hipStream_t s) {
    switch (a.c.D) {
        case 64: return chunk_d<KV, QT, 64>(a, s);
        case 128: return chunk_d<KV, QT, 128>(a, s);
        default: return chunk_d<KV, QT, 256>(a, s);
    }
}

}  // namespace

// Tiles of a part at least, where a request's block is split.
constexpr int kPartTiles = 4;

ChunkPlan chunk_plan(const wb_kv_cache& c, int N, int R, int Hq, int width) {
    const int G = Hq / c.H;
    ChunkPlan p;
    // rows of a block: 128, or 256 where a wavefront's registers hold 64 and requests have as many
    p.rows = 128;
    p.heads = G < p.rows ? G : p.rows;
    p.head_blocks = (G + p.heads - 1) / p.heads;
    p.tokens = p.rows / p.heads;
    p.part_tiles = kPartTiles;
    p.target = 256 * waves_per_simd(c.D, p.rows / 128);
    const int64_t by_tokens = int64_t(N) / p.tokens + R, blocks = (N < by_tokens ? N : by_tokens) * int64_t(c.H) * p.head_blocks;
    const int64_t tiles = (int64_t(width) * c.page + kTile - 1) / kTile;
    p.slots = 0;
    if (tiles > kPartTiles) {
        // (a block of s tiles has ceil(s / t) parts of at most t >= all tiles / target: fewer than
        // 2 s / t where that is more than one)
        const int64_t most = blocks * ((tiles + kPartTiles - 1) / kPartTiles);
        p.slots = most < 2 * p.target ? most : 2 * p.target;
    }
    p.groups = blocks + (p.slots ? p.target : 0);
    p.part_o_bytes = size_t(p.slots) * p.rows * c.D * 4;
    p.part_ml_bytes = size_t(p.slots) * p.rows * 8;
    return p;
}

hipError_t launch_chunk(const ChunkArgs& a, hipStream_t s) {
    if (a.c.dtype == WB_BF16) return chunk_t<WB_BF16, WB_BF16>(a, s);
    if (a.c.dtype == WB_F16) return chunk_t<WB_F16, WB_F16>(a, s);
    return a.q_dtype == WB_BF16 ? chunk_t<WB_E4M3, WB_BF16>(a, s) : chunk_t<WB_E4M3, WB_F16>(a, s);
}

}  // namespace wb
