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
//     Float16 limbs hold 2^15 p, which is at most 2^15: their smallest step, 2^-24, is then
//     2^-39 of the largest weight. (Limbs of p itself lose a weight of e^-17.4 altogether, which
//     is all there is of a row whose one heavy token has a value near 0.)
// Work is split along the cache. Its units are turns of 128 tokens (a tile for each of a
// workgroup's 4 wavefronts) of one request for one block of heads, in the order (request,
// block, turn); as many workgroups as the card holds at once take equal runs of them, found
// from the lengths on the device, so that ragged batches and single long requests fill the
// card alike and captured graphs keep working as lengths grow. A run may cover several
// segments (all turns, or the rest, or the first of a request's block). Segments that are
// whole are finished by their workgroup; the others, at most two a workgroup, leave their sums
// in the caller's workspace, where the workgroup that stores a segment's last part, or a
// second launch, joins them in the order of the cache: results do not depend on timing.
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

// Run of workgroup w of n: units [total w / n, total (w + 1) / n)
__device__ __forceinline__ int64_t run_start(int64_t total, int64_t w, int64_t n) { return quotient64(total * w, n); }
// The workgroup whose run holds unit u
__device__ __forceinline__ int64_t run_of(int64_t total, int64_t u, int64_t n) { return quotient64((u + 1) * n - 1, total); }

struct Run {
    int64_t total, from, to;        // all units; this workgroup's
    int64_t start;                  // first unit of request r
    int r;                          // the request of unit `from`
    int n;                          // workgroups with work
    int lens_at, lens;              // the lane's length of requests lens_at ..+63, r's among them
};

// This workgroup's run (from == to: none), by every wavefront for itself: lane l sums the
// turns of requests [l R / 64, (l + 1) R / 64), one scan finds the lane whose requests hold
// the run's first unit, another the request among them. (Lengths that change under a call give
// wrong results, but every index stays inside: places are clamped.)
__device__ __forceinline__ Run find_run(const AttendArgs& A) {
    const int lane = threadIdx.x & 63;
    const int most = A.width << A.page_log2, per = (A.R + 63) / 64;
    auto len_at = [&](int r) { return r < A.R ? A.lens[r] : 0; };
    auto turns_at = [&](int r, int len) { return r < A.R ? turns_of(len, A.window, most) : 0; };
    const int len0 = len_at(lane);                       // (up to 64 requests: all there is to load)
    int64_t mine = turns_at(lane, len0);
    if (per > 1) {
        mine = 0;
#pragma unroll 4
        for (int i = 0; i < per; ++i) mine += turns_at(lane * per + i, len_at(lane * per + i));
    }
    const int64_t upto = wave_scan(mine);
    Run s;
    s.total = lane64(upto, 63) * A.head_blocks;
    const int n = s.n = int(s.total < gridDim.x ? s.total : int64_t(gridDim.x));
    s.r = s.lens_at = 0;
    s.lens = len0;
    s.from = s.to = s.start = 0;
    if (int(blockIdx.x) >= n) return s;
    s.from = run_start(s.total, blockIdx.x, n);
    s.to = run_start(s.total, int64_t(blockIdx.x) + 1, n);
    const int64_t at = quotient64(s.from, A.head_blocks);          // in turns of all requests before
    const int who = __ffsll((unsigned long long)__ballot(upto > at)) - 1;
    int64_t before = lane64(upto, who) - lane64(mine, who);
    if (per == 1) {
        s.r = who;
        s.start = before * A.head_blocks;
        return s;
    }
    s.r = min((who + 1) * per, A.R) - 1;
    s.start = before * A.head_blocks;
    for (int base = who * per; base < (who + 1) * per; base += 64) {
        const int turns = base + lane < (who + 1) * per ? turns_at(base + lane, len_at(base + lane)) : 0;
        const int64_t sum = before + wave_scan(turns);
        const uint64_t past = __ballot(sum > at);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            s.r = base + l;
            s.start = (lane64(sum, l) - __builtin_amdgcn_readlane(turns, l)) * A.head_blocks;
            break;
        }
        before = lane64(sum, 63);
    }
    s.lens_at = s.r & ~63;
    s.lens = len_at(s.lens_at + lane);
    return s;
}

// Wavefronts a SIMD holds, which is workgroups a compute unit holds. 16 KB of tile in flight a
// wavefront saturate HBM with one each (64 ragged requests of 128 bfloat16 columns: 73.1 us with
// one, 75.6 with two, 85.0 with three); smaller tiles and conversions want more of them. 64
// columns with three, two and one: 256 ragged e4m3 requests to 4096 tokens 91.5, 96.2 and 142 us,
// 100 float16 windows of 1024 tokens 61.0, 61.8 and 77.2, 64 ragged bfloat16 requests 43.8, 42.9
// and 47.1. e4m3 with two and one: 128 columns 153.4 and 176.5 us, 256 columns 91.5 and 95.5 with
// a bfloat16 query, but 118.2 and 106.3 with the two limbs of a float16 one.
constexpr int waves_per_simd(int kv, int qt, int D) {
    if (D == 64) return 3;
    if (kv == WB_E4M3) return D == 128 || qt == WB_BF16 ? 2 : 1;
    return 1;
}

// A place in a run: turn `turn` of request r for block of heads hb
struct Place {
    int r, hb, kvh, turn, turns;    // (turns: of the request; kvh: the block's key-value head)
    int n, from;                    // the request's tokens (0 if its length is bad), the first that is read
    bool bad_len;
};

// 16-bit matrix operands
template <int T>
struct Mat;
template <>
struct Mat<WB_BF16> {
    static __device__ __forceinline__ f32x4 mul(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    }
};
template <>
struct Mat<WB_F16> {
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
    static constexpr float kLimbs = MT == WB_F16 ? 0x1p15f : 1.f;     // what the weights' limbs are multiplied by
    using M = Mat<MT>;

    // q's operands: lane l holds head l % 16, the 8 values that meet the keys' 8 of each product
    static __device__ __forceinline__ void load_q(const AttendArgs& A, int r, int kvh, int qb, u32x4 hi[KQ], u32x4 lo[KQ]) {
        const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
        const int heads = min(16, A.G - 16 * qb), head0 = kvh * A.G + 16 * qb;
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

// 4 columns of a finished row (sum v, weight sum l, maximum m) out to o and lse.
template <int QT>
__device__ __forceinline__ void finish(const AttendArgs& A, f32x4 v, float l, float m, size_t row, int D, int col) {
    const float by = l == 0.f ? 1.f : l;
    u32x2 out;
    out[0] = uint32_t(Elem<QT>::put(v[0] / by)) | uint32_t(Elem<QT>::put(v[1] / by)) << 16;
    out[1] = uint32_t(Elem<QT>::put(v[2] / by)) | uint32_t(Elem<QT>::put(v[3] / by)) << 16;
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(A.o) + row * D + col) = out;
    if (A.lse && col == 0) A.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

// The parts that units [from, to) of one request and block were computed in: `count` (1: they
// were finished by their workgroup) in the slots at(c) of the workspace.
struct Parts {
    int64_t first;
    int w0, count;
    __device__ __forceinline__ Parts(int64_t total, int64_t n, int64_t from, int64_t to) {
        w0 = int(run_of(total, max(from, int64_t(0)), n));
        count = int(run_of(total, min(to, total) - 1, n)) - w0 + 1;
        first = 2 * int64_t(w0) + (run_start(total, w0, n) != from);
    }
    __device__ __forceinline__ size_t at(int c) const { return size_t(c ? 2 * (int64_t(w0) + c) : first); }
};
__device__ __forceinline__ Parts parts_of(const AttendArgs& A, int r, int hb) {
    const int64_t total = A.spans[A.R], start = A.spans[r], end = r + 1 < A.R ? A.spans[r + 1] : total;
    const int64_t turns = quotient64(end - start, A.head_blocks);
    return Parts(total, total < A.groups ? total : A.groups, start + hb * turns, start + (hb + 1) * turns);
}

// Parts that are joined HERE, in the launch that stores them, are stored and loaded at the
// card's scope, past the caches that its compute dies do not share: a wavefront whose stores
// have completed then needs no write-back of its die's cache before others may read them, nor
// they an invalidation of theirs. (With fences, which do both for the whole cache, the batch of
// 64 ragged requests takes 162 us, not 73.)
template <bool HERE>
__device__ __forceinline__ void put_part(float* p, f32x2 v) {
    if constexpr (HERE)
        __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    else
        *reinterpret_cast<f32x2*>(p) = v;
}
template <bool HERE>
__device__ __forceinline__ f32x2 get_part(const float* p) {
    if constexpr (!HERE) return *reinterpret_cast<const f32x2*>(p);
    return __builtin_bit_cast(f32x2, __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                                       __HIP_MEMORY_SCOPE_AGENT));
}
// 4 columns of head h of a row joined from parts c0, c0 + 2^step_log2, ...: their sum, weight sum and
// maximum, in one pass with a running maximum (a part's sums are requested with its maximum)
struct Joined {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    __device__ __forceinline__ void add(f32x4 vc, float mc, float lc) {
        const float top = fmaxf(m, mc), ref = top == -INFINITY ? 0.f : top;
        const float f = __builtin_amdgcn_exp2f(m - ref), fc = __builtin_amdgcn_exp2f(mc - ref);
        l = l * f + lc * fc;
        v = v * f + vc * fc;
        m = top;
    }
};
template <int D, bool HERE>
__device__ __forceinline__ Joined join_columns(const AttendArgs& A, const Parts& parts, int h, int col, int c0,
                                               int step_log2) {
    Joined j;
#pragma unroll 8
    for (int i = 0; i < (parts.count - c0 + (1 << step_log2) - 1) >> step_log2; ++i) {
        const size_t at = parts.at(c0 + (i << step_log2)) * 16 + h;
        const f32x2 ml = get_part<HERE>(A.part_ml + 2 * at), v0 = get_part<HERE>(A.part_o + at * D + col),
                    v1 = get_part<HERE>(A.part_o + at * D + col + 2);
        j.add(f32x4{v0[0], v0[1], v1[0], v1[1]}, ml[0], ml[1]);
    }
    return j;
}

// JOINS: the workgroup that comes last joins a split segment (else a second launch does)
template <int KV, int QT, int D, bool JOINS>
__global__ void __launch_bounds__(kThreads, waves_per_simd(KV, QT, D)) attend_kernel(const AttendArgs A) {
    using T = Attend<KV, QT, D>;
    using M = typename T::M;
    constexpr int KQ = T::KQ, VB = T::VB, VN = T::VN, LD = T::LD;
    // Two sets of a segment's sums where they fit, taken in turn: a wavefront may store the next
    // segment's while others read this one's, and one barrier a segment is enough.
    constexpr int kSets = D == 256 && waves_per_simd(KV, QT, D) == 2 ? 1 : 2;
    __shared__ float sums_[kSets][kWaves][16][LD];
    __shared__ float stat_m_[kSets][kWaves][16], stat_l_[kSets][kWaves][16];
    __shared__ int bad_page_[kSets][kWaves];
    __shared__ int is_last;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int head = lane & 15, g = lane >> 4;
    const int blocks_of_kv = A.head_blocks / A.c.H;
    const int page_mask = (1 << A.page_log2) - 1;
    const float mul = A.scale * kLog2e;
    const Run run = find_run(A);
    if (!JOINS && A.spans && blockIdx.x == 0 && tid == 0) A.spans[A.R] = run.total;
    if (run.from == run.to) return;

    // The run as a sequence of turns. Three places of it are in work at a time: the turn that
    // is computed, the next one, whose keys and values are requested, and the one after it,
    // whose page ids are. Requests' ends make no difference to the sequence: at the start of
    // a request or block the loads have been in flight as long as inside one.
    int lens_at = run.lens_at, lens64 = run.lens;
    Place cur;
    auto enter = [&](Place& p, int r) {
        if (r - lens_at >= 64) {
            lens_at = r & ~63;
            lens64 = lens_at + lane < A.R ? A.lens[lens_at + lane] : 0;
        }
        const int n = __builtin_amdgcn_readlane(lens64, r - lens_at), most = A.width << A.page_log2;
        p.r = r;
        p.bad_len = n < 0 || n > most;
        p.n = p.bad_len ? 0 : n;
        p.turns = turns_of(p.n, A.window, most);
        p.from = first_token(p.n, A.window);
    };
    auto advance = [&](Place& p) {
        if (++p.turn < p.turns) return;
        p.turn = 0;
        if (++p.hb == A.head_blocks) {
            p.hb = 0;
            enter(p, min(p.r + 1, A.R - 1));             // (the run ends before, unless lengths change under it)
        }
        p.kvh = p.hb / blocks_of_kv;
    };
    const int64_t units = run.to - run.from;
    enter(cur, run.r);
    const int64_t in_r = max(run.from - run.start, int64_t(0));
    cur.hb = int(min(quotient64(in_r, cur.turns), int64_t(A.head_blocks) - 1));
    cur.kvh = cur.hb / blocks_of_kv;
    cur.turn = int(min(in_r - int64_t(cur.hb) * cur.turns, int64_t(cur.turns) - 1));
    Place next = cur;
    if (units > 1) advance(next);
    Place after = next;
    if (units > 2) advance(after);

    // First token of the lane's group (8 tokens of a tile, from `off`) at a place, clamped into
    // the request; the page id there; and the row of the stored arrays that holds it: a bad
    // page id is noted and page 0 read instead
    auto token_at = [&](const Place& p, int off) {
        return max(0, min(p.from + p.turn * kTurn + wave * kTile + off, (p.n - 1) & ~7));
    };
    auto page_at = [&](const Place& p, int off) { return A.table[size_t(p.r) * A.width + (token_at(p, off) >> A.page_log2)]; };
    int bad = 0;
    auto row_in = [&](const Place& p, int page, int off) -> size_t {
        const bool ok = page >= 0 && page < A.c.pages;
        bad |= !ok && p.n > 0;
        page = ok && p.n > 0 ? page : 0;
        return ((size_t(page) * A.c.H + p.kvh) << A.page_log2) + (token_at(p, off) & page_mask);
    };

    // A tile's keys and values as they are stored, and the scales of the lane's 8 tokens
    constexpr int KL = KV == WB_E4M3 ? KQ / 2 : KQ;             // 16-byte loads of a key
    constexpr int VW = KV == WB_E4M3 ? VB / 4 : VB / 2;         // words of a value block
    u32x4 kr[2][KL];
    uint32_t vr[VN][8][VW];
    f32x4 ks[2], vs[2];
    const int koff = 8 * (head >> 2), voff = 8 * g;
    auto load_keys = [&](size_t row, size_t row_v) {
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
            const f32x4* s = reinterpret_cast<const f32x4*>(A.c.k_scale + row_v);
            ks[0] = s[0];
            ks[1] = s[1];
        }
    };
    auto load_values = [&](size_t row) {
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

    // (page ids first: the first keys wait for them)
    int pk = page_at(cur, koff), pv = page_at(cur, voff);
    const int pk_next = page_at(next, koff), pv_next = page_at(next, voff);
    u32x4 qh[KQ], ql[KQ];
    T::load_q(A, cur.r, cur.kvh, cur.hb - cur.kvh * blocks_of_kv, qh, ql);
    size_t row_v;
    {
        const size_t row_k = row_in(cur, pk, koff);
        row_v = row_in(cur, pv, voff);
        load_keys(row_k, row_v);
        load_values(row_v);
    }
    pk = pk_next;
    pv = pv_next;

    f32x4 acc[VN * VB];
    float m, l;
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < VN * VB; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        m = -INFINITY;
        l = 0.f;
    };
    clear();
    bool first_segment = true;
    int set = 0;
    int t0 = cur.turn;                                          // of the segment

    for (int64_t k = 0; k < units; ++k) {
            const int n = cur.n, base = cur.from + cur.turn * kTurn + wave * kTile;
            const int seen = A.window && n > A.window ? n - A.window : 0;     // first token that counts
            const bool new_block = next.hb != cur.hb || next.r != cur.r;
            if (!JOINS && A.spans && cur.hb == 0 && cur.turn == 0 && tid == 0) A.spans[cur.r] = run.from + k;

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
            // The next tile's keys, as soon as the scores have taken this one's. (Behind the last
            // tile this is the same tile again, from the caches. Loads return in order: the page
            // ids of the place after are requested before the values of the next, or waiting
            // for them would wait for those too.)
            const int bad_here = bad;
            bad = 0;
            if (new_block) T::load_q(A, next.r, next.kvh, next.hb - next.kvh * blocks_of_kv, qh, ql);
            const size_t row_k = row_in(next, pk, koff);
            row_v = row_in(next, pv, voff);
            load_keys(row_k, row_v);
            pk = page_at(after, koff);
            pv = page_at(after, voff);

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
                a *= T::kLimbs;
                b *= T::kLimbs;
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
            load_values(row_v);

            const bool last_turn = cur.turn + 1 == cur.turns;
            if (last_turn || k + 1 == units) {
    // end of a segment: join the wavefronts
    const bool alone = t0 == 0 && last_turn;
    const int slot = 2 * int(blockIdx.x) + !first_segment;      // of its sums, if it is not whole
    const int r = cur.r, kvh = cur.kvh, qb = cur.hb - kvh * blocks_of_kv;
    const int heads = min(16, A.G - 16 * qb), head0 = kvh * A.G + 16 * qb;
    l = add_xor32_f32(add_xor16_f32(l));
    if (kSets == 1 && !first_segment) __syncthreads();          // (the last segment's have been read)
    auto& sums = sums_[set];
    auto& stat_m = stat_m_[set];
    auto& stat_l = stat_l_[set];
    auto& bad_page = bad_page_[set];
    set = kSets - 1 - set;
    if (g == 0) {
        stat_m[wave][head] = m;
        stat_l[wave][head] = l;
    }
    const int any_bad = __any(bad_here);
    if (lane == 0) bad_page[wave] = any_bad;
    if (head < heads) {
#pragma unroll
        for (int vn = 0; vn < VN; ++vn)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < VB; c += 4) {
                    f32x4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[vn * VB + c + e][i];
                    *reinterpret_cast<f32x4*>(&sums[wave][head][vn * 16 * VB + (4 * g + i) * VB + c]) = v;
                }
    }
    __syncthreads();
    int poison = cur.bad_len;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) poison |= bad_page[w];

    for (int e = tid; e < heads * (D / 4); e += kThreads) {
        const int h = e / (D / 4), d = (e - h * (D / 4)) * 4;
        float mm = stat_m[0][h], ll = 0.f;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, stat_m[w][h]);
        const float ref = mm == -INFINITY ? 0.f : mm;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(stat_m[w][h] - ref);
            v += *reinterpret_cast<const f32x4*>(&sums[w][h][d]) * f;
            ll += stat_l[w][h] * f;
        }
        v *= 1.f / T::kLimbs;
        if (poison) ll = __builtin_nanf("");
        if (alone) {
            finish<QT>(A, v, ll, mm, size_t(r) * A.Hq + head0 + h, D, d);
        } else {
            const size_t at = size_t(slot) * 16 + h;
            put_part<JOINS>(A.part_o + at * D + d, f32x2{v[0], v[1]});
            put_part<JOINS>(A.part_o + at * D + d + 2, f32x2{v[2], v[3]});
            if (d == 0) put_part<JOINS>(A.part_ml + 2 * at, f32x2{mm, ll});
        }
    }

    if (JOINS && !alone) {
        // the workgroup that stores the last part of a segment joins it
        stores_complete();
        __syncthreads();
        const int64_t unit0 = run.from + k - cur.turn;
        const Parts parts(run.total, run.n, unit0, unit0 + cur.turns);
        if (tid == 0) is_last = last_to_arrive(A.arrivals + parts.w0, A.tag, parts.count);
        __syncthreads();
        if (is_last) {
            // a lane per 4 columns, and where lanes are left every `ways`-th part
            const int items = heads * (D / 4);
            int ways_log2 = 0;
            while ((items << (ways_log2 + 1)) <= kThreads && (2 << ways_log2) <= parts.count) ++ways_log2;
            const int ways = 1 << ways_log2;
            const int way = ways > 1 ? tid / items : 0;
            auto row_of = [&](int h) { return size_t(r) * A.Hq + head0 + h; };
            if (ways == 1) {
                for (int e = tid; e < items; e += kThreads) {
                    const int h = e / (D / 4), d = 4 * (e - h * (D / 4));
                    const Joined j = join_columns<D, true>(A, parts, h, d, 0, 0);
                    finish<QT>(A, j.v, j.l, j.m, row_of(h), D, d);
                }
            } else {
                const int e = tid - way * items, h = e / (D / 4), d = 4 * (e - h * (D / 4));
                Joined j;
                // (the sums have been read: their place holds each way's, 8 floats a lane)
                f32x4* place = reinterpret_cast<f32x4*>(&sums[0][0][0]);
                if (way < ways) {
                    j = join_columns<D, true>(A, parts, h, d, way, ways_log2);
                    place[2 * tid] = j.v;
                    place[2 * tid + 1] = f32x4{j.m, j.l, 0.f, 0.f};
                }
                __syncthreads();
                if (way == 0) {
                    for (int w = 1; w < ways; ++w) {
                        const f32x4 ml = place[2 * (w * items + e) + 1];
                        j.add(place[2 * (w * items + e)], ml[0], ml[1]);
                    }
                    finish<QT>(A, j.v, j.l, j.m, row_of(h), D, d);
                }
            }
        }
    }

    clear();
    first_segment = false;
    t0 = next.turn;
            } else {
                bad |= bad_here;
            }
            cur = next;
            next = after;
            if (k + 3 < units) advance(after);
    }
}

// Joins the segments of a request. Few requests (which may have hundreds each): a workgroup
// per (request, query head, 64 columns), 16 lanes across the columns and 16 along the segments.
constexpr int kJoinThreads = 256, kJoinCols = 64;
constexpr int kLongWorkgroups = 2048;
template <int QT, int D>
__global__ void __launch_bounds__(kJoinThreads) join_long_kernel(const AttendArgs A) {
    constexpr int L = kJoinCols / 4, N = kJoinThreads / L;
    static_assert(N == 16, "ways along the segments");
    __shared__ f32x4 sums[N][L];
    __shared__ f32x2 stats[N][L];
    const int r = blockIdx.x, h = blockIdx.y;
    const int kvh = h / A.G, in_kv = h - kvh * A.G;
    const Parts parts = parts_of(A, r, kvh * (A.head_blocks / A.c.H) + in_kv / 16);
    if (parts.count == 1) return;
    const int d = threadIdx.x % L, w = threadIdx.x / L, col = blockIdx.z * kJoinCols + 4 * d;
    Joined j = join_columns<D, false>(A, parts, in_kv & 15, col, w, 4);
    sums[w][d] = j.v;
    stats[w][d] = f32x2{j.m, j.l};
    __syncthreads();
    if (w) return;
#pragma unroll
    for (int i = 1; i < N; ++i) j.add(sums[i][d], stats[i][d][0], stats[i][d][1]);
    finish<QT>(A, j.v, j.l, j.m, size_t(r) * A.Hq + h, D, col);
}

// Many requests (of few segments each, most of them whole, with nothing to join): a workgroup
// per request and block of heads, a lane per 4 columns.
template <int QT, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttendArgs A) {
    const int r = blockIdx.x / A.head_blocks, hb = blockIdx.x - r * A.head_blocks;
    const Parts parts = parts_of(A, r, hb);
    if (parts.count == 1) return;
    const int blocks_of_kv = A.head_blocks / A.c.H;
    const int kvh = hb / blocks_of_kv, qb = hb - kvh * blocks_of_kv;
    const int heads = min(16, A.G - 16 * qb);
    for (int e = threadIdx.x; e < heads * (D / 4); e += kJoinThreads) {
        const int h = e / (D / 4), d = e - h * (D / 4);
        const Joined j = join_columns<D, false>(A, parts, h, 4 * d, 0, 0);
        finish<QT>(A, j.v, j.l, j.m, size_t(r) * A.Hq + kvh * A.G + 16 * qb + h, D, 4 * d);
    }
}

template <int KV, int QT, int D>
hipError_t attend_d(const AttendArgs& a, hipStream_t s) {
    if (a.arrivals) {
        attend_kernel<KV, QT, D, true><<<a.groups, kThreads, 0, s>>>(a);
        return hipGetLastError();
    }
    attend_kernel<KV, QT, D, false><<<a.groups, kThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.spans) return e;
    if (int64_t(a.R) * a.Hq * (D / kJoinCols) <= kLongWorkgroups)
        join_long_kernel<QT, D><<<dim3(a.R, a.Hq, D / kJoinCols), kJoinThreads, 0, s>>>(a);
    else
        join_kernel<QT, D><<<unsigned(a.R) * unsigned(a.head_blocks), kJoinThreads, 0, s>>>(a);
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

// A request's block may get nearly all of its share of the workgroups (their number over that
// of blocks), and the one that comes last joins their parts: above kPartsJoined of them for
// each lane that costs more than a second launch of many workgroups. 32 query and 8 key-value
// heads of 128 columns, joined by the last workgroup / by a second launch: 1 request of 237
// tokens 9.3 / 12.0 us, 1 of 8000 (16 parts a lane) 15.1 / 15.4, 8 to 512 tokens 9.3 / 12.1, 32
// to 1024 17.7 / 21.6, 64 to 4096 73.0 / 74.8; 20 heads of 64 columns, 24 windows of 1024: 20.1
// / 21.6; 1 request of 8000 with 32 query and 4 key-value heads of 256 columns 55.3 / 18.6, with
// 64 query heads (128 parts a lane) 88.2 / 19.7.
constexpr int kPartsJoined = 32;

// As many workgroups as the card's 256 compute units hold at once, and no more than all
// requests at full width have units.
AttendPlan attend_plan(const wb_kv_cache& c, int R, int Hq, int width, int q_dtype) {
    const int G = Hq / c.H;
    AttendPlan p;
    p.head_blocks = c.H * ((G + 15) / 16);
    const int per_cu = waves_per_simd(c.dtype, q_dtype, c.D);
    const int64_t turns = (int64_t(width) * c.page + kTurn - 1) / kTurn;
    const int64_t most = int64_t(R) * turns * p.head_blocks;
    p.groups = int(most < 256 * per_cu ? most : 256 * per_cu);
    p.part_o_bytes = p.part_ml_bytes = p.spans_bytes = p.arrivals_bytes = 0;
    p.joins_itself = false;
    if (turns > 1) {
        const size_t rows = size_t(p.groups) * 2 * 16;
        p.part_o_bytes = rows * c.D * 4;
        p.part_ml_bytes = rows * 8;
        p.spans_bytes = (size_t(R) + 1) * 8;
        p.arrivals_bytes = size_t(p.groups) * 8;
        const int heads = G < 16 ? G : 16;
        p.joins_itself = int64_t(p.groups) * heads * (c.D / 4) <= int64_t(kPartsJoined) * kThreads * p.head_blocks;
    }
    return p;
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t s) {
    if (a.c.dtype == WB_BF16) return attend_t<WB_BF16, WB_BF16>(a, s);
    if (a.c.dtype == WB_F16) return attend_t<WB_F16, WB_F16>(a, s);
    return a.q_dtype == WB_BF16 ? attend_t<WB_E4M3, WB_BF16>(a, s) : attend_t<WB_E4M3, WB_F16>(a, s);
}

}  // namespace wb
