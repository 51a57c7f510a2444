// Log probabilities of given tokens, entropy and the most probable tokens (wbserve.h).
//
//   lse = log sum_j e^{x_j},  logprob = x_token - lse,  entropy = lse - sum_j p_j x_j
//
// Reading the logits once bounds it (HBM; the exponentials and sums take about as long, 9 operations and
// an exponential a column). A workgroup takes a row, or, where rows are few, a segment of one; a lane
// takes vectors of 8 columns and keeps, of d = x log2 e - ref with a whole number ref from the running
// maximum up (or, where that is 2^26 and more, d = (x - maximum) log2 e), s = sum 2^d and t = sum 2^d d. An
// exponent is rounded once, relative to itself, a change of ref is an exact factor, and the entropy is
// log s - t / s. Where one token has nearly all the probability both are about its d, in (-1, 0], and what
// is left of their difference is within 1e-7 or so of a small entropy: less than 0 is returned as 0.
// The top K need no second pass over the row: the stream leaves the maximum of every group of 64, 512 or
// 1024 columns in LDS. K groups by (maximum, then position) hold all of the top K, for any column of
// another group is behind the maxima of K that are larger, or as large and before it. Those groups are
// read again, and columns at or above the least of their maxima kept: a few more than K, as a rule.
// Where they do not fit (constant rows, or all columns but a few at -infinity), the first K of those
// groups' vectors are found likewise, and the top K among their 8 K columns.
// 2047 rows of 151001 bfloat16 logits with 5 alternatives: 121 us, 5.1 TB/s (618 MB), with 64 151; one float32 row of
// 128000 with 20: 13.8 us.
#include "serve_device.hpp"

namespace wb {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kMaxTop = 64, kMaxGroups = 512;
constexpr int kMaxKeys = 4096;                    // in LDS
constexpr int kOrdered = 128;                     // keys that are ordered by comparing all pairs
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kFar = 0x1p26f;                   // references are whole numbers below it

// Order of values as whole numbers: larger ones first, -0 as 0, NaN as -infinity
__device__ __forceinline__ uint32_t order_of(float x) {
    x = x != x ? -INFINITY : x + 0.f;
    const uint32_t b = __float_as_uint(x);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
// Larger values before smaller, equal ones by position. 0 stands for nothing.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t at) { return uint64_t(order_of(x)) << 32 | (0xFFFFFFFFu - at); }
__device__ __forceinline__ uint32_t at_of(uint64_t key) { return 0xFFFFFFFFu - uint32_t(key); }

// A row in vectors of 8 columns from an aligned address on: vector v holds columns 8 v - off ..+7, of which some of
// the first and the last may be outside [0, V).
template <int T>
struct Row {
    static constexpr int kWords = T == WB_F32 ? 8 : 4;
    const void* p;
    int V, off;
    __device__ __forceinline__ float one(int64_t i) const {
        if constexpr (T == WB_F32) return static_cast<const float*>(p)[i];
        else return Elem<T>::get(static_cast<const uint16_t*>(p)[i]);
    }
    // whether vectors [v, v + n) are all inside
    __device__ __forceinline__ bool inside(int64_t v, int n) const { return 8 * v >= off && 8 * (v + n) <= int64_t(V) + off; }
    __device__ __forceinline__ void load(int64_t v, uint32_t (&w)[kWords]) const {
        const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(p) + (8 * v - off) * (T == WB_F32 ? 4 : 2));
        *reinterpret_cast<u32x4*>(w) = s[0];
        if constexpr (T == WB_F32) *reinterpret_cast<u32x4*>(w + 4) = s[1];
    }
    static __device__ __forceinline__ void unpack(const uint32_t (&w)[kWords], float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (T == WB_F32) x[e] = __uint_as_float(w[e]);
            else if constexpr (T == WB_BF16) x[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
            else x[e] = Elem<T>::get(uint16_t(w[e / 2] >> (16 * (e & 1))));
        }
    }
    // -infinity for columns outside, which adds nothing and is never taken
    __device__ __forceinline__ void get(int64_t v, float (&x)[8]) const {
        if (inside(v, 1)) {
            uint32_t w[kWords];
            load(v, w);
            unpack(w, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t i = 8 * v - off + e;
                x[e] = -INFINITY;
                if (i >= 0 && i < V) x[e] = one(i);
            }
        }
    }
};
__device__ __forceinline__ float largest(const float (&x)[8]) {
    float top = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
    return fmaxf(top, -INFINITY);                                  // (NaN throughout)
}

// s and t of another reference, which is `by` (in powers of two) above theirs if that is negative
__device__ __forceinline__ void move_sums(float& s, float& t, float by) {
    // (2^-256 is 0: nothing is left of sums so far below, which the product must not turn into NaN)
    by = fmaxf(by, -256.f);
    const float f = __builtin_amdgcn_exp2f(by);
    t = (t + s * by) * f;
    s *= f;
}
// s = sum 2^{c x - ref}, t = sum 2^{c x - ref} (c x - ref) of a lane's columns and more (ref -infinity: nothing yet)
struct Sums {
    double ref = -INFINITY;
    float s = 0.f, t = 0.f;
    __device__ __forceinline__ void move(double to) {            // to >= ref
        move_sums(s, t, ref == to ? 0.f : float(ref - to));
        ref = to;
    }
    __device__ __forceinline__ void over_lanes() {
        double top;
        if (__any(fabs(ref) >= kFar && ref != -INFINITY)) {
            top = fmax(ref, __shfl_xor(ref, 1));
#pragma unroll
            for (int d = 2; d < 64; d *= 2) top = fmax(top, __shfl_xor(top, d));
        } else {                                                 // (whole numbers that float32 holds)
            top = value_of(lanes_reduce<OpMax, 64>(order_of(float(ref))));
        }
        move(top);
        s = __uint_as_float(lanes_reduce<OpAdd, 64>(__float_as_uint(s)));
        t = __uint_as_float(lanes_reduce<OpAdd, 64>(__float_as_uint(t)));
    }
};

// The places of the K largest of n <= 64 M values, equal ones by their place, by one wavefront: the K-th largest bit by
// bit, with ballots. Returns a bound that they reach and no other value passes, 0 if there are no more than K.
template <int M>
__device__ __forceinline__ uint32_t largest_of(const uint32_t* values, int n, int K, int* places) {
    const int lane = threadIdx.x & 63;
    uint32_t v[M];
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = 64 * i + lane < n ? values[64 * i + lane] : 0;       // (0 is below every value's order)
    uint32_t least = 0;
    int reach = 0;
    for (uint32_t bit = 0x80000000u; bit && reach != K; bit >>= 1) {
        int count = 0;
#pragma unroll
        for (int i = 0; i < M; ++i) count += __popcll(__ballot(v[i] >= (least | bit)));
        if (count >= K) {
            least |= bit;
            reach = count;
        }
    }
    int above = 0;
#pragma unroll
    for (int i = 0; i < M; ++i) above += __popcll(__ballot(v[i] > least));
    int equal = K - above, at = 0;             // of those at the bound, the first
    const uint64_t before = (uint64_t(1) << lane) - 1;
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const uint64_t same = __ballot(v[i] == least);
        const bool take = v[i] > least || (v[i] == least && __popcll(same & before) < equal);
        const uint64_t taken = __ballot(take);
        if (take) places[at + __popcll(taken & before)] = 64 * i + lane;
        at += __popcll(taken);
        equal -= min(equal, int(__popcll(same)));
    }
    return least;
}
__device__ __forceinline__ uint32_t largest_values(const uint32_t* values, int n, int K, int* places) {
    if (n <= K) {
        if (int(threadIdx.x & 63) < n) places[threadIdx.x & 63] = threadIdx.x & 63;          // (K <= 64)
        return 0;
    }
    if (n <= 64) return largest_of<1>(values, n, K, places);
    if (n <= 128) return largest_of<2>(values, n, K, places);
    if (n <= 256) return largest_of<4>(values, n, K, places);
    return largest_of<8>(values, n, K, places);
}

// The first K of n distinct keys (at most kOrdered) in order, out[0 .. K) (0 where there are fewer), by all threads of the
// workgroup, which have all stored their keys
__device__ __forceinline__ void order_keys(const uint64_t* keys, int n, int K, uint64_t* out) {
    // each key's place is the number of larger ones
    const int tid = threadIdx.x;
    for (int i = n + tid; i < K; i += kThreads) out[i] = 0;
    if (tid < n) {
        const uint64_t mine = keys[tid];
        int place = 0;
        const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(keys);
#pragma unroll 8
        for (int j = 0; j < n / 2; ++j) {
            const ulonglong2 k = pairs[j];
            place += (k.x > mine) + (k.y > mine);
        }
        if (n & 1) place += keys[n - 1] > mine;
        if (place < K) out[place] = mine;
    }
    __syncthreads();
}
// The same of any number of keys. `spare` has room for kOrdered of them, `bins` for 256 counts.
__device__ __forceinline__ void first_keys(const uint64_t* keys, int n, int K, uint64_t* out, uint64_t* spare, int* bins) {
    const int tid = threadIdx.x;
    if (n <= kOrdered) return order_keys(keys, n, K, out);
    // Digit by digit, from the highest, the K-th key's; until those at or above its digits are few enough to be ordered
    __shared__ int state[3];                     // its digit; keys above the digits so far; keys taken
    uint64_t prefix = 0;
    int above = 0, shift = 64, at_or_above;
    do {
        shift -= 8;
        __syncthreads();
        if (tid < 256) bins[tid] = 0;
        if (tid == 0) state[2] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads)
            if (shift == 56 || keys[i] >> (shift + 8) == prefix) atomicAdd(&bins[keys[i] >> shift & 255], 1);
        __syncthreads();
        if (tid < 64) {
            // lane l holds digits 255 - 4 l ..252 - 4 l
            int c[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += c[i] = bins[255 - 4 * tid - i];
            int before = int(wave_scan(sum)) - sum + above;
            if (before < K && before + sum >= K) {
                int i = 0;
                while (before + c[i] < K) before += c[i++];
                state[0] = 255 - 4 * tid - i;
                state[1] = before;
            }
        }
        __syncthreads();
        above = state[1];
        prefix = prefix << 8 | uint64_t(state[0]);
        at_or_above = above + bins[state[0]];
    } while (at_or_above > kOrdered);            // (keys differ: behind the last digit those are K)
    for (int i = tid; i < n; i += kThreads)
        if (keys[i] >> shift >= prefix) spare[atomicAdd(&state[2], 1)] = keys[i];
    __syncthreads();
    order_keys(spare, at_or_above, K, out);
}

// Wavefronts a SIMD has room for. Float32 chunks of 1024 columns do not fit the registers of eight: 2000 rows of 100000 with
// 20 alternatives 151 us, 193 with eight (600 rows of 128000 66.1 and 69.5).
constexpr int waves_per_simd(int type, int J) { return type == WB_F32 && J == 2 ? 6 : 8; }

// A wavefront takes chunks of 64 J vectors at a time. TOP: vectors of a group, whose maximum is kept: 8 (64 columns), 64 J
// (a chunk), or 0: no alternatives are wanted.
template <int T, int TOP, int J>
__global__ void __launch_bounds__(kThreads, waves_per_simd(T, J)) logprobs_kernel(const LogprobArgs A) {
    constexpr int kKeys = TOP ? kMaxKeys : 2;
    __shared__ __attribute__((aligned(16))) uint64_t keys[kKeys];
    __shared__ uint64_t first[TOP ? kMaxTop : 1];
    __shared__ __attribute__((aligned(16))) uint64_t spare[TOP ? kOrdered : 2];
    __shared__ uint32_t maxima[TOP ? kMaxGroups : 1];
    __shared__ int group_at[TOP ? kMaxTop : 1];
    __shared__ uint32_t bound;
    __shared__ int bins[TOP ? 256 : 1];
    __shared__ double refs[kWaves];
    __shared__ float sums[kWaves][2];
    __shared__ int count, is_last;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = A.first + blockIdx.x / A.segments;
    const int segment = blockIdx.x % A.segments;
    const int size = T == WB_F32 ? 4 : 2;
    Row<T> x;
    x.p = static_cast<const uint8_t*>(A.logits) + row * A.row * size;
    x.V = A.V;
    x.off = int((reinterpret_cast<uintptr_t>(x.p) & 15) / size);
    const float c = A.scale * kLog2e;
    const int vectors = (A.V + x.off + 7) / 8, chunks = (vectors + 64 * J - 1) / (64 * J);
    const int c0 = int(int64_t(chunks) * segment / A.segments), c1 = int(int64_t(chunks) * (segment + 1) / A.segments);

    // Of the lane, while it reads: s and t about 2^ref (ref a whole number, or -infinity: nothing yet) or, if the
    // wavefront's references have come to kFar, about e^{scale ref}, where ref is a logit
    float ref = -INFINITY, s = 0.f, t = 0.f;
    bool far = false;
    uint32_t next[J][Row<T>::kWords];
    auto fetch = [&](int k) {                           // chunks that are all inside, ahead of their use
        if (k < c1 && x.inside(int64_t(64) * J * k, 64 * J))
#pragma unroll
            for (int j = 0; j < J; ++j) x.load(int64_t(64) * (J * k + j) + lane, next[j]);
    };
    fetch(c0 + wave);
    for (int k = c0 + wave; k < c1; k += kWaves) {
        float y[J][8];
        if (x.inside(int64_t(64) * J * k, 64 * J)) {
#pragma unroll
            for (int j = 0; j < J; ++j) Row<T>::unpack(next[j], y[j]);
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j) x.get(int64_t(64) * (J * k + j) + lane, y[j]);
        }
        fetch(k + kWaves);
        float top = -INFINITY, least = INFINITY;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                top = fmaxf(top, y[j][e]);
                least = fminf(least, y[j][e]);
            }
        // A whole-number reference is a rounded product, which the columns' exact ones pass by up to half of its last
        // place: 2 below kFar, 2^7 and more from 2^31 on, past what the sums hold; and products end at 2^128. Past kFar
        // differences are taken first, from the largest logit.
        const float reach = top * c;
        if (far || __any(!(fabsf(fmaxf(reach, ref)) < kFar))) {
            const bool was = far;
            const float up = was ? fmaxf(reach, ref * c) : fmaxf(reach, ref);
            far = __any(!(fabsf(up) < kFar) && fmaxf(top, ref) > -INFINITY);      // (c x may be -infinity)
            if (far != was) {
                const float to = far ? fmaxf(top, ref * __builtin_amdgcn_rcpf(c)) : ceilf(up);
                move_sums(s, t, far ? __builtin_fmaf(-to, c, ref) : __builtin_fmaf(ref, c, -to));      // (NaN: nothing yet)
                ref = to;
            }
            if (far) {
                if (top > ref) {
                    move_sums(s, t, (ref - top) * c);
                    ref = top;
                }
                const float base = ref == -INFINITY ? 0.f : ref;
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[j][e] -= base;
                least = -INFINITY;
            }
        }
        if (!far && reach > ref) {
            const float to = ceilf(reach);
            move_sums(s, t, ref - to);
            ref = to;
        }
        const float less = far || ref == -INFINITY ? 0.f : -ref;
        if (__any(!(__builtin_fmaf(least, c, less) > -256.f))) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = __builtin_fmaf(y[j][e], c, less), p = __builtin_amdgcn_exp2f(d);
                    s += p;
                    t = __builtin_fmaf(p, fmaxf(d, -256.f), t);     // (0 times -infinity is not 0)
                }
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = __builtin_fmaf(y[j][e], c, less), p = __builtin_amdgcn_exp2f(d);
                    s += p;
                    t = __builtin_fmaf(p, d, t);
                }
        }
        if constexpr (TOP) {
            constexpr int kLanes = TOP / J, kGroups = 64 / kLanes;
            const uint32_t best = lanes_reduce<OpMax, kLanes>(order_of(top)), group = uint32_t(k) * kGroups + lane / kLanes;
            if (lane % kLanes == 0) maxima[group - c0 * kGroups] = best;
        }
    }
    Sums own{far ? double(ref) * c : double(ref), s, t};
    own.over_lanes();
    if (lane == 0) {
        refs[wave] = own.ref;
        sums[wave][0] = own.s;
        sums[wave][1] = own.t;
    }
    if (tid == 0) count = 0;
    __syncthreads();
    own = Sums{};
    if (lane < kWaves) own = Sums{refs[lane], sums[lane][0], sums[lane][1]};
    own.over_lanes();

    if constexpr (TOP) {
        const int K = A.K, n = (c1 - c0) * (64 * J / TOP), held = min(K, n);
        if (wave == 0) {
            const uint32_t least = largest_values(maxima, n, K, group_at);
            if (lane == 0) bound = least;
        }
        __syncthreads();
        const uint32_t least = bound;                                          // no column below it is taken
        const int group0 = c0 * (64 * J / TOP);
        // Columns of those groups, two vectors of a lane on their way at a time (keys past the room are counted, not
        // stored)
        for (int from = 0; from < held * TOP; from += 2 * kThreads) {
            float y[2][8];
            int at[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int i = from + u * kThreads + tid;
                at[u] = A.V;
                if (i < held * TOP) {
                    const int v = TOP * (group0 + group_at[i / TOP]) + i % TOP;
                    x.get(v, y[u]);
                    at[u] = v * 8 - x.off;
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (at[u] < A.V && order_of(largest(y[u])) >= least)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (order_of(y[u][e]) >= least && at[u] + e >= 0 && at[u] + e < A.V) {
                            const int place = atomicAdd(&count, 1);
                            if (place < kKeys) keys[place] = key_of(y[u][e], uint32_t(at[u] + e));
                        }
        }
        __syncthreads();
        const int found = count;
        if (found <= kKeys) {
            first_keys(keys, found, K, first, spare, bins);
        } else {
            // vectors first
            __syncthreads();
            if (tid == 0) count = 0;
            __syncthreads();
            for (int i = tid; i < held * TOP; i += kThreads) {
                const int v = TOP * (group0 + group_at[i / TOP]) + i % TOP;
                float y[8];
                x.get(v, y);
                const uint32_t o = order_of(largest(y));
                if (v < vectors && o >= least) keys[atomicAdd(&count, 1)] = uint64_t(o) << 32 | (0xFFFFFFFFu - uint32_t(v));
            }
            __syncthreads();
            const int n_vectors = count;
            first_keys(keys, n_vectors, K, first, spare, bins);
            if (tid == 0) count = 0;
            uint64_t mine = 0;
            if (tid < 8 * min(K, n_vectors)) {
                const int64_t at = int64_t(at_of(first[tid >> 3])) * 8 - x.off + (tid & 7);
                if (at >= 0 && at < A.V) mine = key_of(x.one(at), uint32_t(at));
            }
            __syncthreads();
            if (mine) keys[atomicAdd(&count, 1)] = mine;
            __syncthreads();
            first_keys(keys, count, K, first, spare, bins);
        }
    }

    if (A.segments > 1) {
        // the workgroup that stores a row's last segment joins them, in their order
        const int64_t local = row - A.first;
        const int parts = A.segments, words = 2 + (TOP ? A.K : 0);
        uint64_t* part = A.parts + (local * parts + segment) * words;
        if (tid == 0) {
            put_word(part, __builtin_bit_cast(uint64_t, own.ref));
            put_word(part + 1, uint64_t(__float_as_uint(own.s)) | uint64_t(__float_as_uint(own.t)) << 32);
        }
        if constexpr (TOP)
            if (tid < A.K) put_word(part + 2 + tid, first[tid]);
        stores_complete();
        __syncthreads();
        if (tid == 0) is_last = last_to_arrive(A.arrivals + local, A.tag, parts);
        __syncthreads();
        if (!is_last) return;
        part = A.parts + local * parts * words;
        Sums all;
        if (lane < parts) {                       // (64 parts at most)
            const uint64_t r = get_word(part + lane * words), st = get_word(part + lane * words + 1);
            all = Sums{__builtin_bit_cast(double, r), __uint_as_float(uint32_t(st)), __uint_as_float(uint32_t(st >> 32))};
        }
        all.over_lanes();
        own = all;
        if constexpr (TOP) {
            for (int i = tid; i < parts * A.K; i += kThreads) {
                const int p = i / A.K;
                keys[i] = get_word(part + p * words + 2 + (i - p * A.K));
                if (i < kMaxGroups) maxima[i] = uint32_t(keys[i] >> 32);
            }
            __syncthreads();
            if (parts * A.K > kMaxGroups) {
                first_keys(keys, parts * A.K, A.K, first, spare, bins);
            } else {
                // (equal values are in the order of their columns here)
                if (wave == 0) largest_values(maxima, parts * A.K, A.K, group_at);
                __syncthreads();
                if (tid < A.K) spare[tid] = keys[group_at[tid]];
                __syncthreads();
                order_keys(spare, A.K, A.K, first);
            }
        }
    }

    // c x - ref - log2 s, in powers of two
    const float log_s = log2f(own.s);
    auto logprob_of = [&](float value) {
        const float lp = float((__builtin_fma(double(value), double(c), -own.ref) - log_s) * 0.6931471805599453);
        return lp > 0.f ? 0.f : lp;                   // (s is rounded; a NaN stays)
    };
    if (tid == 0) {
        const int64_t token = A.wide ? static_cast<const int64_t*>(A.tokens)[row] : static_cast<const int32_t*>(A.tokens)[row];
        A.logprob[row] = token >= 0 && token < A.V ? logprob_of(x.one(token)) : __builtin_nanf("");
        const float entropy = (log_s - own.t / own.s) * kLn2;
        if (A.entropy) A.entropy[row] = entropy < 0.f ? 0.f : entropy;
    }
    if constexpr (TOP)
        if (tid < A.K) {
            A.top_ids[row * A.K + tid] = int32_t(at_of(first[tid]));
            A.top_logprobs[row * A.K + tid] = logprob_of(value_of(uint32_t(first[tid] >> 32)));
        }
}

template <int T>
hipError_t logprobs_t(const LogprobArgs& a, unsigned groups, hipStream_t s) {
    if (!a.K && a.chunk == 1) logprobs_kernel<T, 0, 1><<<groups, kThreads, 0, s>>>(a);
    else if (!a.K) logprobs_kernel<T, 0, 2><<<groups, kThreads, 0, s>>>(a);
    else if (a.group == 8) logprobs_kernel<T, 8, 1><<<groups, kThreads, 0, s>>>(a);
    else if (a.group == 64) logprobs_kernel<T, 64, 1><<<groups, kThreads, 0, s>>>(a);
    else logprobs_kernel<T, 128, 2><<<groups, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// Segments of a row: enough for 256 workgroups, one a compute unit (with four of them a batch of 32 rows of 128000 and 20
// alternatives takes 24.4 us, not 18.0: every segment finds alternatives of its own), of 16 chunks of 512 columns at least,
// and so that their alternatives can be ordered as one list. A segment's groups, whose maxima are kept: the largest of which
// there are twice as many as alternatives wanted (or hardly anything could be left out), up to 512, and whose vectors, of
// the first K groups, fit LDS (K 128 of them up to 32 alternatives; past that K 64, so that 64 segments hold 2^24 - 8
// columns from any alignment on).
LogprobPlan logprob_plan(int N, int V, int K) {
    const int chunks = (V + 7 + 511) / 512;
    LogprobPlan p;
    int64_t n = 256 / N < 1 ? 1 : 256 / N;
    if (n > chunks / 16) n = chunks / 16 < 1 ? 1 : chunks / 16;
    if (n > 64) n = 64;
    if (K && n > kMaxGroups / K) n = kMaxGroups / K;
    const bool wide = K * 128 <= kMaxKeys;
    const int64_t room = wide ? 2 * kMaxGroups : kMaxGroups, least = (chunks + room - 1) / room;
    if (n < least) n = least;
    const int64_t c = (chunks + n - 1) / n;
    p.group = wide && c / 2 >= 2 * K ? 128 : c >= 2 * K || c > kMaxGroups / 8 ? 64 : 8;
    p.chunk = K ? (p.group == 128 ? 2 : 1) : c >= 256 ? 2 : 1;
    p.segments = int(n);
    p.part_bytes = n > 1 ? size_t(N) * n * (2 + K) * 8 : 0;
    p.arrivals_bytes = n > 1 ? size_t(N) * 8 : 0;
    return p;
}

hipError_t launch_logprobs(LogprobArgs a, int N, hipStream_t s) {
    const int64_t most = kLaunchItems / kThreads / a.segments;            // rows of a launch
    uint64_t* const parts = a.parts;
    uint64_t* const arrivals = a.arrivals;
    for (int64_t first = 0; first < N; first += most) {
        const int64_t n = N - first < most ? N - first : most;
        a.first = first;
        if (a.segments > 1) {
            a.parts = parts + first * a.segments * (2 + a.K);
            a.arrivals = arrivals + first;
        }
        const unsigned groups = unsigned(n * a.segments);
        const hipError_t e = a.dtype == WB_BF16  ? logprobs_t<WB_BF16>(a, groups, s)
                             : a.dtype == WB_F16 ? logprobs_t<WB_F16>(a, groups, s)
                                                 : logprobs_t<WB_F32>(a, groups, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace wb
