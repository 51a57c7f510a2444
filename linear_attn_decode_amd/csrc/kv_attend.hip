// Attention of one new token per request over a paged key-value cache (wbserve.h).
//
//   o = sum_t e^{s_t - m} v_t / sum_t e^{s_t - m},  s_t = scale q . k_t,  m = max s_t
//
// in one pass over the stored tokens with a running maximum. Reading K and V once bounds it
// (HBM); the products are a few percent of the matrix cores' rate even with the query heads
// of a key-value head padded to 16. What the layout is chosen for is that keys and values go
// from HBM into matrix operands without LDS, lane exchanges or barriers:
//   * A wavefront takes tiles of 32 tokens. Scores are K Q^T by 16x16x32 products: operand A
//     (lane l: row l % 16, 8 contiguous values) is 16 bytes of token row l % 16 as stored, B
//     the 16 query heads. Row m of half t of the tile is token 8 (m / 4) + 4 t + m % 4, so
//     that the result (lane l: head l % 16, rows 4 (l / 16) ..+3 of both halves) leaves each
//     lane with the scores of the 8 consecutive tokens 8 (l / 16) ..+7.
//   * Those 8 weights are, in place, operand B of the product with the values (lane l:
//     column = head l % 16, 8 contraction steps of group l / 16). Operand A then has to hold
//     8 tokens of one value column: a lane loads 16 bytes (columns 8 (l % 16) ..+7) of its
//     group's 8 tokens and transposes the 8 x 8 block in its own registers by byte permutes
//     (half an operation per value). Product c takes column c of every lane's block, so its
//     result (lane l: head l % 16, rows 4 (l / 16) ..+3) is columns 8 (4 (l / 16) + r) + c:
//     over all c each lane ends with contiguous columns of its head.
//   * The weights enter as two 16-bit limbs, p = hi + lo: the second product costs matrix
//     time that is idle anyway and keeps their rounding (2^-9 in bfloat16) out of the result.
// Work is split along the cache: a workgroup (4 wavefronts, 128 tokens a turn) takes a chunk
// of one request's tokens for one key-value head. The chunk length follows from the lengths
// on the device (every workgroup sums them), so that ragged batches and single long requests
// fill the card alike and captured graphs keep working as lengths grow. A request of one
// chunk is finished by its workgroup; others leave their sums in the caller's workspace for
// a second, small launch.
#include "serve_device.hpp"

namespace wb {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, kTile = 32, kTurn = kTile * kWaves;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// First token read of a request of n tokens (n >= 0), at the start of its group of 8
__device__ __forceinline__ int first_token(int n, int window) {
    return window && n > window ? (n - window) & ~7 : 0;
}
// Turns of 128 tokens of a request; a request without tokens (or with a bad length, which
// only gets its NaN) takes one
__device__ __forceinline__ int turns_of(int n, int window, int most) {
    if (n <= 0 || n > most) return 1;
    return (n - first_token(n, window) + kTurn - 1) / kTurn;
}

struct Span {
    int r, first, count, index;     // request, its first chunk, its chunks, this chunk among them
    int turns;
};

// The request that chunk x works for (r < 0: none) -- by every wavefront for itself, 64
// requests at a time.
__device__ __forceinline__ Span find_span(const AttendArgs& A, int x) {
    const int lane = threadIdx.x & 63;
    const int most = A.width << A.page_log2;
    int64_t total = 0;
    for (int base = 0; base < A.R; base += 64) {
        const int r = base + lane;
        total += r < A.R ? turns_of(A.lens[r], A.window, most) : 0;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d, 64);
    // turns of a chunk: as many as spread all turns over `target` workgroups
    const int64_t each64 = (total * A.head_blocks + A.target - 1) / A.target;
    const int each = int(each64 < 1 ? 1 : each64);
    Span s{-1, 0, 0, 0, 0};
    int before = 0;
    for (int base = 0; base < A.R; base += 64) {
        const int r = base + lane;
        const int turns = r < A.R ? turns_of(A.lens[r], A.window, most) : 0;
        const int count = (turns + each - 1) / each;
        const int upto = before + wave_scan(count);
        const uint64_t past = __ballot(upto > x);
        if (past) {
            const int who = __ffsll((unsigned long long)past) - 1;
            s.r = base + who;
            s.count = __shfl(count, who, 64);
            s.first = __shfl(upto, who, 64) - s.count;
            s.turns = __shfl(turns, who, 64);
            s.index = x - s.first;
            break;
        }
        before = __shfl(upto, 63, 64);
    }
    return s;
}

// 16-bit matrix operands
template <int T>
struct Mat;
template <>
struct Mat<WB_BF16> {
    typedef bf16x8 V8;
    static __device__ __forceinline__ f32x4 mul(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    }
};
template <>
struct Mat<WB_F16> {
    typedef f16x8 V8;
    static __device__ __forceinline__ f32x4 mul(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
    }
};

// Two bfloat16 values (exact) of bytes 0, 1 or 2, 3 of four e4m3 codes
template <bool HIGH>
__device__ __forceinline__ uint32_t e4m3_to_bf16x2(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
}

// KV: the cache's type; QT: the type of q and o. MT, the operands' type, is the cache's, and
// bfloat16 for an 8-bit cache (whose codes it holds exactly); a float16 q then enters as two
// limbs, which hold it exactly too.
template <int KV, int QT, int D>
struct Attend {
    static constexpr int MT = KV == WB_E4M3 ? WB_BF16 : KV;
    static constexpr bool kTwoQ = KV == WB_E4M3 && QT == WB_F16;
    static constexpr int KQ = D / 32;                 // score products of a half tile
    static constexpr int VB = D == 64 ? 4 : 8;        // value columns of a lane's block
    static constexpr int VN = D / (16 * VB);          // blocks of a lane (2 for D = 256)
    static constexpr int LD = D + 4;                  // LDS stride of a head's sums
    using M = Mat<MT>;

    // q's operands: lane l holds head l % 16, the 8 values that meet the keys' 8 of each product
    static __device__ __forceinline__ void load_q(const AttendArgs& A, int r, int head0, int heads, u32x4 hi[KQ],
                                                  u32x4 lo[KQ]) {
        const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
        const uint16_t* q = static_cast<const uint16_t*>(A.q) + int64_t(r) * A.q_row + int64_t(head0 + n) * A.q_head;
#pragma unroll
        for (int i = 0; i < KQ; ++i) {
            // 8-bit rows are read 16 codes a lane: products 2 j, 2 j + 1 take their halves
            const int d = KV == WB_E4M3 ? 64 * (i / 2) + 16 * g + 8 * (i & 1) : 32 * i + 8 * g;
            u32x4 w = {0, 0, 0, 0};
            if (n < heads) w = *reinterpret_cast<const u32x4*>(q + d);
            if constexpr (!kTwoQ) {
                hi[i] = w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = Elem<WB_F16>::get(uint16_t(w[j])), b = Elem<WB_F16>::get(uint16_t(w[j] >> 16));
                    const uint16_t ah = Elem<WB_BF16>::put(a), bh = Elem<WB_BF16>::put(b);
                    hi[i][j] = uint32_t(ah) | uint32_t(bh) << 16;
                    lo[i][j] = uint32_t(Elem<WB_BF16>::put(a - Elem<WB_BF16>::get(ah))) |
                               uint32_t(Elem<WB_BF16>::put(b - Elem<WB_BF16>::get(bh))) << 16;
                }
            }
        }
    }
};

// Wavefronts a SIMD is to hold: a tile in flight of 256 columns takes more than half the registers
template <int KV, int QT, int D>
constexpr int kWavesPerSimd = D == 256 && (KV != WB_E4M3 || QT == WB_F16) ? 1 : 2;

template <int KV, int QT, int D>
__global__ void __launch_bounds__(kThreads, (kWavesPerSimd<KV, QT, D>)) attend_kernel(const AttendArgs A) {
    using T = Attend<KV, QT, D>;
    using M = typename T::M;
    constexpr int KQ = T::KQ, VB = T::VB, VN = T::VN, LD = T::LD;
    __shared__ float sums[kWaves][16][LD];
    __shared__ float stat_m[kWaves][16], stat_l[kWaves][16];
    __shared__ int bad_page[kWaves];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int head = lane & 15, g = lane >> 4;
    // heads vary fastest: the workgroups that run together read whole pages, all heads of them
    // (one head's rows of every page lie in the same few memory channels)
    const int chunk = blockIdx.x / A.head_blocks, hb = blockIdx.x - chunk * A.head_blocks;
    const int blocks_of_kv = A.head_blocks / A.c.H;
    const int kvh = hb / blocks_of_kv, qb = hb - kvh * blocks_of_kv;
    const int heads = min(16, A.G - 16 * qb);                   // query heads of this workgroup
    const int head0 = kvh * A.G + 16 * qb;

    const Span sp = find_span(A, chunk);
    if (sp.r < 0) return;
    const int n = A.lens[sp.r];
    const bool bad_len = n < 0 || n > (A.width << A.page_log2);
    const int from = first_token(n, A.window);                  // first token that is read
    const int seen = A.window && n > A.window ? n - A.window : 0;   // first token that counts
    const int t0 = int(int64_t(sp.turns) * sp.index / sp.count), t1 = int(int64_t(sp.turns) * (sp.index + 1) / sp.count);

    u32x4 qh[KQ], ql[KQ];
    T::load_q(A, sp.r, head0, heads, qh, ql);

    f32x4 acc[VN * VB];
#pragma unroll
    for (int i = 0; i < VN * VB; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    int bad = 0;
    const float mul = A.scale * kLog2e;
    const int32_t* pages = A.table + size_t(sp.r) * A.width;
    const int page_mask = (1 << A.page_log2) - 1;

    // Page of the 8 tokens from t (clamped into the request), and the row of the stored arrays
    // that holds them (a bad page id is noted and page 0 read instead)
    auto page_at = [&](int t) { return pages[min(t, (n - 1) & ~7) >> A.page_log2]; };
    auto row_in = [&](int page, int t) -> size_t {
        if (page < 0 || page >= A.c.pages) {
            bad = 1;
            page = 0;
        }
        return ((size_t(page) * A.c.H + kvh) << A.page_log2) + (min(t, (n - 1) & ~7) & page_mask);
    };

    // A tile's keys and values as they are stored, and the scales of the lane's 8 tokens. The
    // keys of the next tile are requested as soon as the scores have taken this one's, its
    // values behind the product with this one's, its page ids a tile earlier: a wavefront
    // keeps a tile in flight while it computes.
    constexpr int KL = KV == WB_E4M3 ? KQ / 2 : KQ;             // 16-byte loads of a key
    constexpr int VW = KV == WB_E4M3 ? VB / 4 : VB / 2;         // words of a value block
    u32x4 kr[2][KL];
    uint32_t vr[VN][8][VW];
    f32x4 ks[2], vs[2];
    const int koff = 8 * (head >> 2), voff = 8 * g;
    auto load_keys = [&](int page, int page_v, int base) {
        const size_t row = row_in(page, base + koff);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const size_t at = (row + 4 * t + (head & 3)) * D;
            if constexpr (KV == WB_E4M3) {
                const uint8_t* k = static_cast<const uint8_t*>(A.c.k) + at + 16 * g;
#pragma unroll
                for (int i = 0; i < KL; ++i) kr[t][i] = *reinterpret_cast<const u32x4*>(k + 64 * i);
            } else {
                const uint16_t* k = static_cast<const uint16_t*>(A.c.k) + at + 8 * g;
#pragma unroll
                for (int i = 0; i < KL; ++i) kr[t][i] = *reinterpret_cast<const u32x4*>(k + 32 * i);
            }
        }
        if constexpr (KV == WB_E4M3) {
            const f32x4* s = reinterpret_cast<const f32x4*>(A.c.k_scale + row_in(page_v, base + voff));
            ks[0] = s[0];
            ks[1] = s[1];
        }
    };
    auto load_values = [&](int page, int base) {
        const size_t row = row_in(page, base + voff);
#pragma unroll
        for (int vn = 0; vn < VN; ++vn)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const size_t at = (row + j) * D + vn * 16 * VB + head * VB;
                const uint8_t* v = static_cast<const uint8_t*>(A.c.v) + at * (KV == WB_E4M3 ? 1 : 2);
                if constexpr (VW == 4) {
                    *reinterpret_cast<u32x4*>(vr[vn][j]) = *reinterpret_cast<const u32x4*>(v);
                } else if constexpr (VW == 2) {
                    *reinterpret_cast<u32x2*>(vr[vn][j]) = *reinterpret_cast<const u32x2*>(v);
                } else {
                    vr[vn][j][0] = *reinterpret_cast<const uint32_t*>(v);
                }
            }
        if constexpr (KV == WB_E4M3) {
            const f32x4* s = reinterpret_cast<const f32x4*>(A.c.v_scale + row);
            vs[0] = s[0];
            vs[1] = s[1];
        }
    };

    const int end = min(n, from + t1 * kTurn);                   // (n > 0 where it is used)
    int base = from + t0 * kTurn + wave * kTile;
    if (!bad_len && n > 0 && base < end) {
        int pk = page_at(base + koff), pv = page_at(base + voff);
        int pk_next = page_at(base + kTurn + koff), pv_next = page_at(base + kTurn + voff);
        load_keys(pk, pv, base);
        load_values(pv, base);
        for (; base < end; base += kTurn) {
            // (the last tile requests itself again, from the caches: a condition around the
            // loads would make the waits below cover them)
            const int next = base + kTurn < end ? base + kTurn : base;

            // scores: s[t][i] of token base + 8 g + 4 t + i
            f32x4 s[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    const u32x4 w = kr[t][i];
                    if constexpr (KV == WB_E4M3) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const u32x4 a = {e4m3_to_bf16x2<false>(w[2 * e]), e4m3_to_bf16x2<true>(w[2 * e]),
                                             e4m3_to_bf16x2<false>(w[2 * e + 1]), e4m3_to_bf16x2<true>(w[2 * e + 1])};
                            s[t] = M::mul(a, qh[2 * i + e], s[t]);
                            if constexpr (T::kTwoQ) s[t] = M::mul(a, ql[2 * i + e], s[t]);
                        }
                    } else {
                        s[t] = M::mul(w, qh[i], s[t]);
                    }
                }
            }
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = s[j >> 2][j & 3] * mul;
                if constexpr (KV == WB_E4M3) x[j] *= ks[j >> 2][j & 3];
            }
            // (loads return in order: the page ids of the tile after next are requested before
            // the values of the next, or waiting for them would wait for those too)
            if (next != base) {
                pk = pk_next;
                pv = pv_next;
            }
            load_keys(pk, pv, next);
            pk_next = page_at(next + kTurn + koff);
            pv_next = page_at(next + kTurn + voff);

            const bool whole = base >= seen && base + kTile <= n;
            const int tok = base + 8 * g;
            if (!whole) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (tok + j < seen || tok + j >= n) {
                        x[j] = -INFINITY;
                        if constexpr (KV == WB_E4M3) vs[j >> 2][j & 3] = 0.f;
#pragma unroll
                        for (int vn = 0; vn < VN; ++vn)          // 0 * NaN is not 0
#pragma unroll
                            for (int c = 0; c < VW; ++c) vr[vn][j][c] = 0;
                    }
            }

            // running maximum of the head (its 4 lanes agree), weights in two limbs
            float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
            top = max_xor32(max_xor16(top));
            if (__any(top > m)) {
                const float m_new = fmaxf(m, top);
                const float keep = m_new == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - m_new);
                l *= keep;
#pragma unroll
                for (int i = 0; i < VN * VB; ++i) acc[i] *= keep;
                m = m_new;
            }
            const float ref = m == -INFINITY ? 0.f : m;
            u32x4 ph, pl;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a = __builtin_amdgcn_exp2f(x[2 * j] - ref), b = __builtin_amdgcn_exp2f(x[2 * j + 1] - ref);
                l += a + b;
                if constexpr (KV == WB_E4M3) {
                    a *= vs[j >> 1][(2 * j) & 3];
                    b *= vs[j >> 1][(2 * j + 1) & 3];
                }
                const uint16_t ah = Elem<T::MT>::put(a), bh = Elem<T::MT>::put(b);
                ph[j] = uint32_t(ah) | uint32_t(bh) << 16;
                pl[j] = uint32_t(Elem<T::MT>::put(a - Elem<T::MT>::get(ah))) |
                        uint32_t(Elem<T::MT>::put(b - Elem<T::MT>::get(bh))) << 16;
            }

            // values
#pragma unroll
            for (int vn = 0; vn < VN; ++vn)
#pragma unroll
                for (int c2 = 0; c2 < VB / 2; ++c2) {              // a pair of columns
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if constexpr (KV == WB_E4M3)
                            w[j] = c2 & 1 ? e4m3_to_bf16x2<true>(vr[vn][j][c2 / 2]) : e4m3_to_bf16x2<false>(vr[vn][j][c2 / 2]);
                        else
                            w[j] = vr[vn][j][c2];
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t sel = e ? 0x07060302u : 0x05040100u;
                        u32x4 a;
#pragma unroll
                        for (int j = 0; j < 4; ++j) a[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], sel);
                        f32x4& s4 = acc[vn * VB + 2 * c2 + e];
                        s4 = M::mul(a, ph, s4);
                        s4 = M::mul(a, pl, s4);
                    }
                }
            load_values(pv, next);
        }
    }

    // join the wavefronts: everything relative to the workgroup's maximum
    l = add_xor32_f32(add_xor16_f32(l));
    if (g == 0) {
        stat_m[wave][head] = m;
        stat_l[wave][head] = l;
    }
    bad = __any(bad);
    if (lane == 0) bad_page[wave] = bad;
    __syncthreads();
    float M_ = stat_m[0][head];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) M_ = fmaxf(M_, stat_m[w][head]);
    const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - M_);
    if (head < heads) {
#pragma unroll
        for (int vn = 0; vn < VN; ++vn)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < VB; c += 4) {
                    f32x4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[vn * VB + c + e][i] * f;
                    *reinterpret_cast<f32x4*>(&sums[wave][head][vn * 16 * VB + (4 * g + i) * VB + c]) = v;
                }
    }
    __syncthreads();
    int poison = bad_len;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) poison |= bad_page[w];

    const bool alone = sp.count == 1;
    for (int e = tid; e < heads * (D / 4); e += kThreads) {
        const int h = e / (D / 4), d = (e - h * (D / 4)) * 4;
        float mm = stat_m[0][h], ll = 0.f;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, stat_m[w][h]);
        const float ref = mm == -INFINITY ? 0.f : mm;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            v += *reinterpret_cast<const f32x4*>(&sums[w][h][d]);
            ll += stat_l[w][h] * __builtin_amdgcn_exp2f(stat_m[w][h] - ref);
        }
        if (poison) ll = __builtin_nanf("");
        if (alone) {
            const float by = ll == 0.f ? 1.f : ll;
            uint16_t* o = static_cast<uint16_t*>(A.o) + (size_t(sp.r) * A.Hq + head0 + h) * D + d;
            u32x2 w;
            w[0] = uint32_t(Elem<QT>::put(v[0] / by)) | uint32_t(Elem<QT>::put(v[1] / by)) << 16;
            w[1] = uint32_t(Elem<QT>::put(v[2] / by)) | uint32_t(Elem<QT>::put(v[3] / by)) << 16;
            *reinterpret_cast<u32x2*>(o) = w;
            if (A.lse && d == 0) A.lse[size_t(sp.r) * A.Hq + head0 + h] = ll == 0.f ? -INFINITY : mm * kLn2 + logf(ll);
        } else {
            const size_t at = (size_t(chunk) * A.head_blocks + hb) * 16 + h;
            *reinterpret_cast<f32x4*>(A.part_o + at * D + d) = v;
            if (d == 0) {
                A.part_ml[2 * at] = mm;
                A.part_ml[2 * at + 1] = ll;
            }
        }
    }
    if (A.spans && hb == 0 && sp.index == 0 && tid == 0) {
        A.spans[2 * sp.r] = sp.first;
        A.spans[2 * sp.r + 1] = sp.count;
    }
}

// One lane's 4 columns of the joined row (sum v, weight sum l, maximum m) out to o and lse.
template <int QT>
__device__ __forceinline__ void finish(const AttendArgs& A, f32x4 v, float l, float m, size_t row, int D, int col) {
    const float by = l == 0.f ? 1.f : l;
    u32x2 out;
    out[0] = uint32_t(Elem<QT>::put(v[0] / by)) | uint32_t(Elem<QT>::put(v[1] / by)) << 16;
    out[1] = uint32_t(Elem<QT>::put(v[2] / by)) | uint32_t(Elem<QT>::put(v[3] / by)) << 16;
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(A.o) + row * D + col) = out;
    if (A.lse && col == 0) A.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

// Joins the chunks of a request. Few requests (which may have hundreds of chunks each): a
// workgroup per (request, query head, 64 columns), 16 lanes across the columns and 16 along
// the chunks, whose factors are worked out once in LDS.
constexpr int kJoinThreads = 256, kJoinCols = 64, kJoinStep = 1024;
constexpr int kLongWorkgroups = 2048;
template <int QT, int D>
__global__ void __launch_bounds__(kJoinThreads) join_long_kernel(const AttendArgs A) {
    constexpr int NT = kJoinThreads, L = kJoinCols / 4, N = NT / L;
    __shared__ float factor[kJoinStep];
    __shared__ f32x4 part[N][L];
    __shared__ float red_m[NT / 64], red_l[NT / 64];
    const int tid = threadIdx.x;
    const int r = blockIdx.x, h = blockIdx.y;
    const int first = A.spans[2 * r], count = A.spans[2 * r + 1];
    if (count == 1) return;
    const int kvh = h / A.G, in_kv = h - kvh * A.G;
    const int hb = kvh * (A.head_blocks / A.c.H) + in_kv / 16;
    const size_t at0 = (size_t(first) * A.head_blocks + hb) * 16 + (in_kv & 15);
    const size_t step = size_t(A.head_blocks) * 16;

    float m = -INFINITY;
    for (int c = tid; c < count; c += NT) m = fmaxf(m, A.part_ml[2 * (at0 + c * step)]);
    m = max_xor32(max_xor16(m));
#pragma unroll
    for (int d = 8; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    if ((tid & 63) == 0) red_m[tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red_m[0], red_m[1]), fmaxf(red_m[2], red_m[3]));
    const float ref = m == -INFINITY ? 0.f : m;

    const int d = tid % L, w = tid / L;
    const float* col = A.part_o + at0 * D + blockIdx.z * kJoinCols + 4 * d;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
    for (int base = 0; base < count; base += kJoinStep) {
        const int upto = min(kJoinStep, count - base);
        __syncthreads();
        for (int c = tid; c < upto; c += NT) {
            const size_t at = at0 + (base + c) * step;
            const float f = __builtin_amdgcn_exp2f(A.part_ml[2 * at] - ref);
            factor[c] = f;
            l += A.part_ml[2 * at + 1] * f;
        }
        __syncthreads();
#pragma unroll 8
        for (int c = w; c < upto; c += N) v += *reinterpret_cast<const f32x4*>(col + (base + c) * step * D) * factor[c];
    }
    l = __uint_as_float(lanes_reduce<OpAdd, 64>(__float_as_uint(l)));
    if ((tid & 63) == 0) red_l[tid >> 6] = l;
    part[w][d] = v;
    __syncthreads();
    if (w) return;
#pragma unroll
    for (int i = 1; i < N; ++i) v += part[i][d];
    l = (red_l[0] + red_l[1]) + (red_l[2] + red_l[3]);
    finish<QT>(A, v, l, m, size_t(r) * A.Hq + h, D, blockIdx.z * kJoinCols + 4 * d);
}

// Many requests (of few chunks each, most of them one, which has nothing to join): a
// workgroup per request and block of heads, a lane per 4 columns.
template <int QT, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttendArgs A) {
    const int r = blockIdx.x, hb = blockIdx.y;
    const int first = A.spans[2 * r], count = A.spans[2 * r + 1];
    if (count == 1) return;
    const int blocks_of_kv = A.head_blocks / A.c.H;
    const int kvh = hb / blocks_of_kv, qb = hb - kvh * blocks_of_kv;
    const int heads = min(16, A.G - 16 * qb);
    const size_t step = size_t(A.head_blocks) * 16;
    for (int e = threadIdx.x; e < heads * (D / 4); e += kJoinThreads) {
        const int h = e / (D / 4), d = e - h * (D / 4);
        const size_t at0 = (size_t(first) * A.head_blocks + hb) * 16 + h;
        const float* ml = A.part_ml + 2 * at0;
        const float* col = A.part_o + at0 * D + 4 * d;
        float m = -INFINITY;
#pragma unroll 4
        for (int c = 0; c < count; ++c) m = fmaxf(m, ml[2 * c * step]);
        const float ref = m == -INFINITY ? 0.f : m;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        float l = 0.f;
#pragma unroll 4
        for (int c = 0; c < count; ++c) {
            const float f = __builtin_amdgcn_exp2f(ml[2 * c * step] - ref);
            l += ml[2 * c * step + 1] * f;
            v += *reinterpret_cast<const f32x4*>(col + c * step * D) * f;
        }
        finish<QT>(A, v, l, m, size_t(r) * A.Hq + kvh * A.G + 16 * qb + h, D, 4 * d);
    }
}

template <int KV, int QT, int D>
hipError_t attend_d(const AttendArgs& a, hipStream_t s) {
    attend_kernel<KV, QT, D><<<unsigned(a.chunks) * unsigned(a.head_blocks), kThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.spans) return e;
    if (int64_t(a.R) * a.Hq * (D / kJoinCols) <= kLongWorkgroups)
        join_long_kernel<QT, D><<<dim3(a.R, a.Hq, D / kJoinCols), kJoinThreads, 0, s>>>(a);
    else
        join_kernel<QT, D><<<dim3(a.R, a.head_blocks), kJoinThreads, 0, s>>>(a);
    return hipGetLastError();
}
template <int KV, int QT>
hipError_t attend_t(const AttendArgs& a, hipStream_t s) {
    switch (a.c.D) {
        case 64: return attend_d<KV, QT, 64>(a, s);
        case 128: return attend_d<KV, QT, 128>(a, s);
        default: return attend_d<KV, QT, 256>(a, s);
    }
}

}  // namespace

constexpr int kTarget = 1024;
// Chunks: `target` workgroups fill the card; R more because every request rounds its own up,
// and never more than all requests at full width have turns.
AttendPlan attend_plan(const wb_kv_cache& c, int R, int Hq, int width) {
    const int G = Hq / c.H;
    AttendPlan p;
    p.head_blocks = c.H * ((G + 15) / 16);
    p.target = kTarget;
    const int64_t turns = (int64_t(width) * c.page + kTurn - 1) / kTurn;
    const int64_t spread = (p.target + p.head_blocks - 1) / p.head_blocks + R;
    const int64_t most = int64_t(R) * turns;
    p.chunks = int(most < spread ? most : spread);
    p.part_o_bytes = p.part_ml_bytes = p.spans_bytes = 0;
    if (turns > 1) {
        const size_t rows = size_t(p.chunks) * p.head_blocks * 16;
        p.part_o_bytes = rows * c.D * 4;
        p.part_ml_bytes = rows * 8;
        p.spans_bytes = (size_t(R) * 8 + 15) / 16 * 16;
    }
    return p;
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t s) {
    if (a.c.dtype == WB_BF16) return attend_t<WB_BF16, WB_BF16>(a, s);
    if (a.c.dtype == WB_F16) return attend_t<WB_F16, WB_F16>(a, s);
    return a.q_dtype == WB_BF16 ? attend_t<WB_E4M3, WB_BF16>(a, s) : attend_t<WB_E4M3, WB_F16>(a, s);
}

}  // namespace wb
