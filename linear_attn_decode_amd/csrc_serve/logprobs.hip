// Log probabilities of given tokens, entropy and the most probable tokens (wbserve.h).
//
//   lse = log sum_j e^{x_j},  logprob = x_token - lse,  entropy = lse - sum_j p_j x_j
//
// Reading the logits once bounds it (HBM; the exponentials and sums take about as long, 9 operations and
// an exponential a column). A workgroup takes a row, or, where rows are few, a segment of one; a lane
// takes vectors of 8 columns and keeps, of d = x log2 e - ref with a whole number ref from the running
// maximum up, s = sum 2^d and t = sum 2^d d. An exponent is rounded once, relative to itself, a change of
// ref is an exact factor, and the entropy is log s - t / s without cancellation.
// The top K need no second pass over the row: the stream leaves the maximum of every chunk of 512 or
// 1024 columns in LDS. K chunks by (maximum, then position) hold all of the top K, for any column of
// another chunk is behind the maxima of K that are larger, or as large and before it. Those chunks are
// read again, and columns at or above the least of their maxima kept: a few more than K, as a rule.
// Where they do not fit (constant rows, or all columns but a few at -infinity), the first K of those
// chunks' vectors are found likewise, and the top K among their 8 K columns.
#include "serve_device.hpp"

namespace wb {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kMaxTop = 64;
constexpr int kMaxKeys = 4096;                    // in LDS
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

// s = sum 2^{c x - ref}, t = sum 2^{c x - ref} (c x - ref), ref a whole number (-infinity: nothing yet)
struct Sums {
    float ref = -INFINITY, s = 0.f, t = 0.f;
    __device__ __forceinline__ void move(float to) {            // to >= ref
        // (2^-256 is 0: nothing is left of sums so far below, which the product must not turn into NaN)
        const float by = ref == to ? 0.f : fmaxf(ref - to, -256.f), f = __builtin_amdgcn_exp2f(by);
        t = (t + s * by) * f;
        s *= f;
        ref = to;
    }
    __device__ __forceinline__ void add(const Sums& o) {
        const float top = fmaxf(ref, o.ref);
        Sums q = o;
        move(top);
        q.move(top);
        s += q.s;
        t += q.t;
    }
};

// The first K of n keys in order, out[0 .. K) (0 where there are fewer), by all threads of the
// workgroup; `keys` has room for the next power of two past n and is left in any order.
__device__ __forceinline__ void first_keys(uint64_t* keys, int n, int K, uint64_t* out) {
    const int tid = threadIdx.x;
    if (n <= kThreads) {
        // each key's place is the number of larger ones
        for (int i = tid; i < K; i += kThreads)
            if (i >= n) out[i] = 0;
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
        return;
    }
    int size = 2 * kThreads;
    while (size < n) size *= 2;
    for (int i = n + tid; i < size; i += kThreads) keys[i] = 0;
    __syncthreads();
    for (int run = 2; run <= size; run *= 2)
        for (int step = run / 2; step; step /= 2) {
            for (int i = tid; i < size / 2; i += kThreads) {
                const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
                const uint64_t a = keys[lo], b = keys[hi];
                if ((a < b) == ((lo & run) == 0)) {
                    keys[lo] = b;
                    keys[hi] = a;
                }
            }
            __syncthreads();
        }
    for (int i = tid; i < K; i += kThreads) out[i] = keys[i];
    __syncthreads();
}

// J: vectors of a lane in a chunk, which is what a wavefront takes at a time
template <int T, bool TOP, int J>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs A) {
    constexpr int kKeys = TOP ? kMaxKeys : 2;
    __shared__ __attribute__((aligned(16))) uint64_t keys[kKeys];
    __shared__ uint64_t first[TOP ? kMaxTop : 1];
    __shared__ float sums[kWaves][3];
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

    Sums own;
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
        if (top * c > own.ref) own.move(ceilf(top * c));
        const float less = own.ref == -INFINITY ? 0.f : -own.ref;
        if (__any(!(__builtin_fmaf(least, c, less) > -256.f))) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = __builtin_fmaf(y[j][e], c, less), p = __builtin_amdgcn_exp2f(d);
                    own.s += p;
                    own.t = __builtin_fmaf(p, fmaxf(d, -256.f), own.t);     // (0 times -infinity is not 0)
                }
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = __builtin_fmaf(y[j][e], c, less), p = __builtin_amdgcn_exp2f(d);
                    own.s += p;
                    own.t = __builtin_fmaf(p, d, own.t);
                }
        }
        if constexpr (TOP) {
            const uint32_t best = lanes_reduce<OpMax, 64>(order_of(top));
            if (lane == 0) keys[k - c0] = uint64_t(best) << 32 | (0xFFFFFFFFu - uint32_t(k));
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        Sums o;
        o.ref = __shfl_xor(own.ref, d);
        o.s = __shfl_xor(own.s, d);
        o.t = __shfl_xor(own.t, d);
        own.add(o);
    }
    if (lane == 0) {
        sums[wave][0] = own.ref;
        sums[wave][1] = own.s;
        sums[wave][2] = own.t;
    }
    if (tid == 0) count = 0;
    __syncthreads();
    own = Sums{sums[0][0], sums[0][1], sums[0][2]};
#pragma unroll
    for (int w = 1; w < kWaves; ++w) own.add(Sums{sums[w][0], sums[w][1], sums[w][2]});

    if constexpr (TOP) {
        const int K = A.K, n = c1 - c0, held = min(K, n);
        first_keys(keys, n, K, first);
        const uint32_t least = n >= K ? uint32_t(first[K - 1] >> 32) : 0;      // no column below it is taken
        // columns of those chunks (keys past the room are counted, not stored)
        for (int i = wave; i < held * J; i += kWaves) {
            const int v = 64 * (J * int(at_of(first[i / J])) + i % J) + lane;
            float y[8];
            x.get(v, y);
            if (v < vectors && order_of(largest(y)) >= least)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int64_t at = int64_t(v) * 8 - x.off + e;
                    if (order_of(y[e]) >= least && at >= 0 && at < A.V) {
                        const int place = atomicAdd(&count, 1);
                        if (place < kKeys) keys[place] = key_of(y[e], uint32_t(at));
                    }
                }
        }
        __syncthreads();
        const int found = count;
        if (found <= kKeys) {
            first_keys(keys, found, K, first);
        } else {
            // vectors first
            __syncthreads();
            if (tid == 0) count = 0;
            __syncthreads();
            for (int i = wave; i < held * J; i += kWaves) {
                const int v = 64 * (J * int(at_of(first[i / J])) + i % J) + lane;
                float y[8];
                x.get(v, y);
                const uint32_t o = order_of(largest(y));
                if (v < vectors && o >= least) keys[atomicAdd(&count, 1)] = uint64_t(o) << 32 | (0xFFFFFFFFu - uint32_t(v));
            }
            __syncthreads();
            const int n_vectors = count;
            first_keys(keys, n_vectors, K, first);
            if (tid == 0) count = 0;
            uint64_t mine = 0;
            if (tid < 8 * min(K, n_vectors)) {
                const int64_t at = int64_t(at_of(first[tid >> 3])) * 8 - x.off + (tid & 7);
                if (at >= 0 && at < A.V) mine = key_of(x.one(at), uint32_t(at));
            }
            __syncthreads();
            if (mine) keys[atomicAdd(&count, 1)] = mine;
            __syncthreads();
            first_keys(keys, count, K, first);
        }
    }

    if (A.segments > 1) {
        // the workgroup that stores a row's last segment joins them, in their order
        const int64_t local = row - A.first;
        const int parts = A.segments, words = 2 + (TOP ? A.K : 0);
        uint64_t* part = A.parts + (local * parts + segment) * words;
        if (tid == 0) {
            put_word(part, uint64_t(__float_as_uint(own.ref)) | uint64_t(__float_as_uint(own.s)) << 32);
            put_word(part + 1, uint64_t(__float_as_uint(own.t)));
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
        for (int p = 0; p < parts; ++p) {
            const uint64_t ms = get_word(part + p * words), t = get_word(part + p * words + 1);
            Sums o;
            o.ref = __uint_as_float(uint32_t(ms));
            o.s = __uint_as_float(uint32_t(ms >> 32));
            o.t = __uint_as_float(uint32_t(t));
            all.add(o);
        }
        own = all;
        if constexpr (TOP) {
            for (int i = tid; i < parts * A.K; i += kThreads) {
                const int p = i / A.K;
                keys[i] = get_word(part + p * words + 2 + (i - p * A.K));
            }
            __syncthreads();
            first_keys(keys, parts * A.K, A.K, first);
        }
    }

    // c x - ref - log2 s, in powers of two (a logit whose c x leaves float32's range: by itself)
    const float log_s = log2f(own.s);
    auto logprob_of = [&](float value) {
        const float d = __builtin_fmaf(value, c, own.ref == -INFINITY ? 0.f : -own.ref) - log_s;
        return fabsf(d) == INFINITY && fabsf(value) < INFINITY ? value * A.scale : d * kLn2;
    };
    if (tid == 0) {
        const int64_t token = A.wide ? static_cast<const int64_t*>(A.tokens)[row] : static_cast<const int32_t*>(A.tokens)[row];
        A.logprob[row] = token >= 0 && token < A.V ? logprob_of(x.one(token)) : __builtin_nanf("");
        if (A.entropy) A.entropy[row] = (log_s - own.t / own.s) * kLn2;
    }
    if constexpr (TOP)
        if (tid < A.K) {
            A.top_ids[row * A.K + tid] = int32_t(at_of(first[tid]));
            A.top_logprobs[row * A.K + tid] = logprob_of(value_of(uint32_t(first[tid] >> 32)));
        }
}

template <int T>
hipError_t logprobs_t(const LogprobArgs& a, unsigned groups, hipStream_t s) {
    if (a.K && a.chunk == 1) logprobs_kernel<T, true, 1><<<groups, kThreads, 0, s>>>(a);
    else if (a.K) logprobs_kernel<T, true, 2><<<groups, kThreads, 0, s>>>(a);
    else if (a.chunk == 1) logprobs_kernel<T, false, 1><<<groups, kThreads, 0, s>>>(a);
    else logprobs_kernel<T, false, 2><<<groups, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// Segments of a row: enough for 1024 workgroups (4 a compute unit), of 32 chunks at least, and of 3 K / 2 where
// alternatives are wanted (with K chunks or fewer in a segment nothing could be left out); joined parts' keys fit LDS,
// and so do a segment's chunks. Chunks of 512 columns where rows are split, so that segments can be short; of 1024
// where a workgroup has a whole row, for half the maxima.
LogprobPlan logprob_plan(int N, int V, int K) {
    const int chunks = (V + 7 + 511) / 512;
    LogprobPlan p;
    int64_t n = 1024 / N < 1 ? 1 : 1024 / N;
    const int64_t most = chunks / (3 * K / 2 > 32 ? 3 * K / 2 : 32);
    if (n > most) n = most < 1 ? 1 : most;
    if (n > 64) n = 64;
    const int64_t least = (chunks + kMaxKeys - 1) / kMaxKeys;
    if (n < least) n = least;
    p.chunk = n > 1 || chunks < 128 ? 1 : 2;
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
