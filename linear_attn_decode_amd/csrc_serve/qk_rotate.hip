// Norms and rotary positions of queries and keys in one pass (wbserve.h).
//
//   y = x / sqrt(mean x^2 + eps) w,   (a, b) -> (a cos t - b sin t, a sin t + b cos t) magnitude,
//   t = position * frequency of the pair
//
// Each value is read and written once, which bounds it (HBM; 32773 tokens of 40 heads of 128, bfloat16: 146 us, 4.58
// TB/s, where a copy reaches 4.76). A wavefront takes one token and
// some of its heads: its lanes find the cosines and sines of the token's angles, one or two
// pairs each, and share them through LDS; then each slot of `lanes` neighbouring lanes takes a
// head at a time, a lane both members of W pairs (or 2 W columns that are not turned), so that
// a head stays in registers between its sum of squares, its rotation and its store.
// Angles are taken in turns and in 64 bits, position * (frequency / 2 pi) less the nearest whole
// number: in 32 bits a position of 10^6 would be off by 0.06 radians.
#include "serve_device.hpp"

namespace wb {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kPairs = 512;                    // of a head at most (1024 columns)

// W values as they are stored, loaded and stored as widely as their alignment (W elements, at most 16 bytes) allows
template <int T, int W>
struct Vec {
    static constexpr int N = T == WB_F32 ? W : (W + 1) / 2;
    uint32_t w[N];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        if constexpr (T == WB_F32) {
            const uint32_t* s = static_cast<const uint32_t*>(p) + at;
            if constexpr (W == 1) w[0] = s[0];
            else
#pragma unroll
                for (int i = 0; i < W; i += 4) *reinterpret_cast<u32x4*>(w + i) = *reinterpret_cast<const u32x4*>(s + i);
        } else {
            const uint16_t* s = static_cast<const uint16_t*>(p) + at;
            if constexpr (W == 8) *reinterpret_cast<u32x4*>(w) = *reinterpret_cast<const u32x4*>(s);
            else if constexpr (W == 4) *reinterpret_cast<u32x2*>(w) = *reinterpret_cast<const u32x2*>(s);
            else w[0] = s[0];
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (T == WB_F32) return __uint_as_float(w[i]);
        else return Elem<T>::get(uint16_t(w[i / 2] >> (16 * (i & 1))));
    }
    template <bool PAST>
    static __device__ __forceinline__ void store(void* p, int64_t at, const float (&x)[W]) {
        if constexpr (T == WB_F32) {
            float* d = static_cast<float*>(p) + at;
            if constexpr (W == 1) d[0] = x[0];
            else
#pragma unroll
                for (int i = 0; i < W; i += 4) put<PAST>(f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]}, d + i);
        } else {
            uint16_t* d = static_cast<uint16_t*>(p) + at;
            if constexpr (W == 1) {
                d[0] = Elem<T>::put(x[0]);
            } else {
                uint32_t w[W / 2];
#pragma unroll
                for (int i = 0; i < W / 2; ++i)
                    w[i] = uint32_t(Elem<T>::put(x[2 * i])) | uint32_t(Elem<T>::put(x[2 * i + 1])) << 16;
                if constexpr (W == 8) put<PAST>(*reinterpret_cast<const u32x4*>(w), d);
                else put<PAST>(*reinterpret_cast<const u32x2*>(w), d);
            }
        }
    }
    template <bool PAST, typename V>
    static __device__ __forceinline__ void put(V v, void* d) {
        if constexpr (PAST) __builtin_nontemporal_store(v, static_cast<V*>(d));
        else *static_cast<V*>(d) = v;
    }
};

// Sum and maximum over slots of 4 to 64 neighbouring lanes
template <typename OP>
__device__ __forceinline__ uint32_t slot_reduce(uint32_t v, int lanes) {
    v = OP::of(v, dpp_u32<0xB1>(v));
    v = OP::of(v, dpp_u32<0x4E>(v));
    if (lanes >= 8) v = OP::of(v, dpp_u32<0x141>(v));
    if (lanes >= 16) v = OP::of(v, dpp_u32<0x140>(v));
    if (lanes >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = OP::of(p[0], p[1]);
    }
    if (lanes >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = OP::of(p[0], p[1]);
    }
    return v;
}

// U: units (W pairs) of a lane, at `lanes` units' distance; PAST: outputs are stored past the caches
template <int T, int W, int U, bool PAST>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateArgs A) {
    __shared__ float table[kWaves][2][kPairs];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t at = int64_t(blockIdx.x) * kWaves + wave;
    const int64_t token = A.first + at / A.waves_per_token;
    if (token >= A.last) return;
    const int part = int(at % A.waves_per_token);
    const int half = A.rot >> 1;
    const int64_t position = A.wide ? static_cast<const int64_t*>(A.positions)[token] : static_cast<const int32_t*>(A.positions)[token];
    float* cosines = table[wave][0];
    float* sines = table[wave][1];
    for (int i = lane; i < half; i += 64) {
        const double turns = double(position) * (A.freqs[i] * 0.15915494309189533577);
        float s, c;
        sincospif(2.f * float(turns - __builtin_rint(turns)), &s, &c);
        cosines[i] = c * A.magnitude;
        sines[i] = s * A.magnitude;
    }
    // (the wavefront's own part of LDS: its stores are ahead of its loads)
    __builtin_amdgcn_wave_barrier();

    const int slots = 64 / A.lanes, slot = lane / A.lanes, in = lane - slot * A.lanes;
    const int turned = half / W, units = (A.D + 2 * W - 1) / (2 * W);
    int c0[U], c1[U];                    // first columns of the unit's two vectors (D: there is none)
    float cs[U][W], sn[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int unit = in + u * A.lanes;
        c0[u] = unit < turned && !A.interleaved ? W * unit : 2 * W * unit;
        if (unit >= units) c0[u] = A.D;
        c1[u] = unit < turned && !A.interleaved ? half + W * unit : c0[u] + W;
        if (c1[u] > A.D - W) c1[u] = A.D;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            cs[u][i] = unit < turned ? cosines[W * unit + i] : 1.f;
            sn[u][i] = unit < turned ? sines[W * unit + i] : 0.f;
        }
    }
    // The weights of queries and keys stay in registers, the next head's columns are on their way behind this one's
    const int heads = A.q.H + A.k.H, step = A.waves_per_token * slots;
    Vec<T, W> wq[2][U], wk[2][U], next[2][U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = i ? c1[u] : c0[u];
            wq[i][u].clear();
            wk[i][u].clear();
            if (c < A.D && A.q.weight) wq[i][u].load(A.q.weight, c);
            if (c < A.D && A.k.weight) wk[i][u].load(A.k.weight, c);
        }
    auto fetch = [&](int head) {
        const bool is_k = head >= A.q.H;
        const void* x = is_k ? A.k.x : A.q.x;
        const int64_t from = is_k ? token * A.k.row + int64_t(head - A.q.H) * A.k.head : token * A.q.row + int64_t(head) * A.q.head;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            next[0][u].clear();
            next[1][u].clear();
            if (head < heads && c0[u] < A.D) next[0][u].load(x, from + c0[u]);
            if (head < heads && c1[u] < A.D) next[1][u].load(x, from + c1[u]);
        }
    };
    fetch(part * slots + slot);
    for (int head = part * slots + slot; head < heads; head += step) {
        const bool is_k = head >= A.q.H;
        const wb_heads& x = is_k ? A.k : A.q;
        const int64_t to = token * x.out_row + int64_t(is_k ? head - A.q.H : head) * x.out_head;
        float a[U][W], b[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                a[u][i] = next[0][u].get(i);
                b[u][i] = next[1][u].get(i);
            }
        fetch(head + step);
        if (x.weight) {
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < W; ++i) sum += a[u][i] * a[u][i] + b[u][i] * b[u][i];
            sum = __uint_as_float(slot_reduce<OpAdd>(__float_as_uint(sum), A.lanes));
            const float mean = sum / float(A.D);
            float by = 1.f / sqrtf(mean + A.eps);
            // Squares that leave float32's range, or lose bits in it: the row is taken times a
            // power of two, its norm in 64 bits
            if (!(mean + A.eps >= 0x1p-100f) || !(mean < INFINITY)) {
                uint32_t top = 0;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < W; ++i) top = max(top, max(magnitude(a[u][i]), magnitude(b[u][i])));
                top = slot_reduce<OpMax>(top, A.lanes);
                if (top == 0) {
                    by = 0.f;                       // (a row of zeros, without eps too)
                } else if (top < 0x7F800000u) {
                    int e;
                    frexpf(__uint_as_float(top), &e);
                    double s = 0.;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            a[u][i] = ldexpf(a[u][i], -e);
                            b[u][i] = ldexpf(b[u][i], -e);
                            s += double(a[u][i]) * a[u][i] + double(b[u][i]) * b[u][i];
                        }
                    const float part_sum = __uint_as_float(slot_reduce<OpAdd>(__float_as_uint(float(s)), A.lanes));
                    by = float(1. / sqrt(double(part_sum) / A.D + ldexp(double(A.eps), -2 * e)));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    a[u][i] = a[u][i] * by * (is_k ? wk[0][u] : wq[0][u]).get(i);
                    b[u][i] = b[u][i] * by * (is_k ? wk[1][u] : wq[1][u]).get(i);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (in + u * A.lanes < turned) {
                float c[W], d[W];
                if (W > 1 && A.interleaved) {
#pragma unroll
                    for (int i = 0; i < W; ++i) {         // pair i: columns 2 i, 2 i + 1 of both vectors together
                        const float p = 2 * i < W ? a[u][(2 * i) % W] : b[u][(2 * i) % W];
                        const float r = 2 * i < W ? a[u][(2 * i + 1) % W] : b[u][(2 * i + 1) % W];
                        const float y0 = __builtin_fmaf(p, cs[u][i], -(r * sn[u][i]));
                        const float y1 = __builtin_fmaf(p, sn[u][i], r * cs[u][i]);
                        (2 * i < W ? c : d)[(2 * i) % W] = y0;
                        (2 * i < W ? c : d)[(2 * i + 1) % W] = y1;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        c[i] = __builtin_fmaf(a[u][i], cs[u][i], -(b[u][i] * sn[u][i]));
                        d[i] = __builtin_fmaf(a[u][i], sn[u][i], b[u][i] * cs[u][i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    a[u][i] = c[i];
                    b[u][i] = d[i];
                }
            }
            if (c0[u] < A.D) Vec<T, W>::template store<PAST>(x.out, to + c0[u], a[u]);
            if (c1[u] < A.D) Vec<T, W>::template store<PAST>(x.out, to + c1[u], b[u]);
        }
    }
}

template <int T>
hipError_t rotate_t(const RotateArgs& a, int W, int units, unsigned groups, hipStream_t s) {
    if (W == 8 && a.past) rotate_kernel<T, 8, 1, true><<<groups, kThreads, 0, s>>>(a);
    else if (W == 8) rotate_kernel<T, 8, 1, false><<<groups, kThreads, 0, s>>>(a);
    else if (W == 4 && a.past) rotate_kernel<T, 4, 1, true><<<groups, kThreads, 0, s>>>(a);
    else if (W == 4) rotate_kernel<T, 4, 1, false><<<groups, kThreads, 0, s>>>(a);
    else if (units <= 64) rotate_kernel<T, 1, 1, false><<<groups, kThreads, 0, s>>>(a);
    else rotate_kernel<T, 1, 8, false><<<groups, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// Elements of a lane's vectors: 8, or 4, if heads and their turned part are whole pairs of such vectors, every
// address and stride is aligned to them and 64 lanes hold a head; else columns one by one.
int rotate_vector(const RotateArgs& a) {
    const int size = a.dtype == WB_F32 ? 4 : 2;
    for (int W = 8; W >= 4; W /= 2) {
        const uintptr_t bytes = uintptr_t(W * size < 16 ? W * size : 16);
        bool ok = a.D % (2 * W) == 0 && a.rot % (2 * W) == 0 && a.D / (2 * W) <= 64;
        for (const wb_heads* x : {&a.q, &a.k}) {
            if (!x->H) continue;
            ok = ok && uintptr_t(x->x) % bytes == 0 && uintptr_t(x->out) % bytes == 0 && uintptr_t(x->weight) % bytes == 0;
            for (const int64_t n : {x->row, x->head, x->out_row, x->out_head}) ok = ok && (n * size) % int64_t(bytes) == 0;
        }
        if (ok) return W;
    }
    return 1;
}

hipError_t launch_rotate(RotateArgs a, int N, hipStream_t s) {
    const int W = rotate_vector(a), units = (a.D + 2 * W - 1) / (2 * W);
    a.lanes = 4;
    while (a.lanes < units && a.lanes < 64) a.lanes *= 2;
    // Wavefronts of a token: one takes all of its heads, which then share its angles, where there are tokens enough for
    // 4096 of them (4 a SIMD); else more, down to one head a slot. (40 heads of 128: 4000 tokens 18.6 us, 20.2 with 8192
    // and 17.5 with 2048; 1000 tokens 6.7, 6.8 and 7.4; column by column, 4000 tokens 46, 53 and 67.)
    const int slots = 64 / a.lanes, rounds = (a.q.H + a.k.H + slots - 1) / slots;
    int64_t wanted = (4096 + int64_t(N) - 1) / N;
    a.waves_per_token = int(wanted < rounds ? wanted : rounds);
    // Outputs that the 256 MB last-level cache could not hold are stored past the caches (32773 tokens of 40 heads of 128,
    // 336 MB: 146 us against 153); what fits is left there for the calls that read it.
    a.past = int64_t(N) * (a.q.H + a.k.H) * a.D * (a.dtype == WB_F32 ? 4 : 2) > int64_t(256) << 20;
    const int64_t most = kLaunchItems / (64 * int64_t(a.waves_per_token));      // tokens of a launch
    for (int64_t first = 0; first < N; first += most) {
        a.first = first;
        a.last = first + most < N ? first + most : N;
        const int64_t waves = (a.last - a.first) * a.waves_per_token;
        const unsigned groups = unsigned((waves + kWaves - 1) / kWaves);
        const hipError_t e = a.dtype == WB_BF16  ? rotate_t<WB_BF16>(a, W, units, groups, s)
                             : a.dtype == WB_F16 ? rotate_t<WB_F16>(a, W, units, groups, s)
                                                 : rotate_t<WB_F32>(a, W, units, groups, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace wb
