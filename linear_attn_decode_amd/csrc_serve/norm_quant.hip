// Root-mean-square norm with the residual's addition and an e4m3 output (wbserve.h).
//
// One pass: a row's h = x + residual stays in registers (8 columns a chunk, V chunks a lane)
// between the sum of squares, the groups' maxima and the codes, so every input is read once
// and every output written once; HBM bounds it (a single row: the launch). The 128 columns
// of a group are 16 neighbouring lanes of one chunk, so a group's maximum is four DPP steps.
// Rows of up to 512 columns take 8, 16, 32 or 64 lanes, several rows a wavefront; wider ones a
// workgroup of as many wavefronts as their chunks need, two chunks a lane (8191 rows of 5000
// bfloat16 columns with a residual: 60.2 us, 4.78 TB/s, the rate of a copy; 68 us with one
// chunk, 65 with three, 73 with four; 2 us less with stores past the caches, but 8192 rows of
// 4096 and the two kernels that read their outputs next then take 78.9 us together, not 74.4). Strides and alignment are free: the
// 16-byte accesses need only the element's alignment on this hardware, and the chunk that
// holds a row's ragged end goes by 4, 2 and 1 columns (bfloat16 with a residual: 400000 rows of
// 100 columns 78.5 us, 109 by single elements; 2352941 rows of 17 174 us, and 305 by single
// elements with 16 lanes a row; 312500 rows of 128 53.1 us).
#include "serve_device.hpp"

namespace wb {
namespace {

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef f32x2 f32x2_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint16_t u16_a1 __attribute__((aligned(1)));

// 8 columns from `at`, or the n < 8 that are left of the row (then 0): 4, 2 and 1 of them by the
// bits of n, three accesses where single elements would be up to seven
template <int T>
__device__ __forceinline__ void load_chunk(const void* p, int64_t at, int n, float x[8]) {
    if constexpr (T == WB_F32) {
        const float* s = static_cast<const float*>(p) + at;
        f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
        if (n >= 8) {
            a = *reinterpret_cast<const f32x4_a4*>(s);
            b = *reinterpret_cast<const f32x4_a4*>(s + 4);
        } else {
            f32x2 pair = {0.f, 0.f};
            float one = 0.f;
            if (n & 4) a = *reinterpret_cast<const f32x4_a4*>(s);
            if (n & 2) pair = *reinterpret_cast<const f32x2_a4*>(s + (n & 4));
            if (n & 1) one = s[n & 6];
            f32x4 rest = {0.f, 0.f, 0.f, 0.f};               // what follows the four
            if (n & 2) rest = f32x4{pair[0], pair[1], one, 0.f};
            else rest[0] = one;
            if (n & 4) b = rest;
            else a = rest;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = a[i];
            x[4 + i] = b[i];
        }
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(p) + at;
        u32x4 w = {0, 0, 0, 0};
        if (n >= 8) {
            w = *reinterpret_cast<const u32x4_a2*>(s);
        } else {
            u32x2 four = {0, 0};
            uint32_t pair = 0, one = 0;
            if (n & 4) four = *reinterpret_cast<const u32x2_a2*>(s);
            if (n & 2) pair = *reinterpret_cast<const u32_a2*>(s + (n & 4));
            if (n & 1) one = s[n & 6];
            const uint32_t r0 = n & 2 ? pair : one, r1 = n & 2 ? one : 0;
            w = n & 4 ? u32x4{four[0], four[1], r0, r1} : u32x4{r0, r1, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = Elem<T>::get(uint16_t(w[i]));
            x[2 * i + 1] = Elem<T>::get(uint16_t(w[i] >> 16));
        }
    }
}

template <int T>
__device__ __forceinline__ void store_chunk(void* p, int64_t at, int n, const float x[8]) {
    if constexpr (T == WB_F32) {
        float* s = static_cast<float*>(p) + at;
        const f32x4 a = {x[0], x[1], x[2], x[3]}, b = {x[4], x[5], x[6], x[7]};
        if (n >= 8) {
            *reinterpret_cast<f32x4_a4*>(s) = a;
            *reinterpret_cast<f32x4_a4*>(s + 4) = b;
        } else {
            const f32x4 rest = n & 4 ? b : a;
            if (n & 4) *reinterpret_cast<f32x4_a4*>(s) = a;
            if (n & 2) *reinterpret_cast<f32x2_a4*>(s + (n & 4)) = f32x2{rest[0], rest[1]};
            if (n & 1) s[n & 6] = n & 2 ? rest[2] : rest[0];
        }
    } else {
        uint16_t* s = static_cast<uint16_t*>(p) + at;
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = uint32_t(Elem<T>::put(x[2 * i])) | uint32_t(Elem<T>::put(x[2 * i + 1])) << 16;
        if (n >= 8) {
            *reinterpret_cast<u32x4_a2*>(s) = w;
        } else {
            const uint32_t r0 = n & 4 ? w[2] : w[0], r1 = n & 4 ? w[3] : w[1];
            if (n & 4) *reinterpret_cast<u32x2_a2*>(s) = u32x2{w[0], w[1]};
            if (n & 2) *reinterpret_cast<u32_a2*>(s + (n & 4)) = r0;
            if (n & 1) s[n & 6] = uint16_t(n & 2 ? r1 : r0);
        }
    }
}

__device__ __forceinline__ void store_codes(uint8_t* s, int n, u32x2 w) {
    if (n >= 8) {
        *reinterpret_cast<u32x2_a1*>(s) = w;
    } else {
        const uint32_t rest = n & 4 ? w[1] : w[0];
        if (n & 4) *reinterpret_cast<u32_a1*>(s) = w[0];
        if (n & 2) *reinterpret_cast<u16_a1*>(s + (n & 4)) = uint16_t(rest);
        if (n & 1) s[n & 6] = uint8_t(n & 2 ? rest >> 16 : rest);
    }
}

// What z is multiplied by for its codes: 448 / most, most = max |z|, in two floats (2^-44 of it),
// so that a code's quotient is rounded once before its own rounding. (8000 rows of 500 bfloat16
// columns: 439 of 4 million codes differ from those of 64 bits, 658 with y, the scale and the
// quotient rounded one after the other; most are exact ties.) 2^-7: the reciprocal of a `most`
// near either end of the range is a normal number.
struct Factor {
    float hi, lo;
};
__device__ __forceinline__ Factor codes_of(float most, float frac, float scale) {
    const float rcp = __builtin_amdgcn_rcpf(most * 0x1p-7f);
    Factor by;
    by.hi = 3.5f * rcp;
    by.lo = __builtin_fmaf(-by.hi, most, kE4M3Max) * 0x1p-7f * rcp;
    if (!(scale > 0x1p-126f && scale < INFINITY)) {
        by.lo = 0.f;
        by.hi = scale == 0x1p-126f ? frac * 0x1p126f     // the smallest scale: not 448 / most
                : scale == 0.f     ? 1.f                 // zeros
                                   : __builtin_nanf("");
    }
    return by;
}

// LR: lanes of a row (8, 16, 32, 64), or 0 for the whole workgroup. V: chunks of a lane.
template <int T, int LR, int V>
__global__ void __launch_bounds__(LR ? 256 : 1024) norm_kernel(const NormArgs A) {
    __shared__ uint32_t red[16];
    const int lanes = LR ? LR : int(blockDim.x);
    const int lane = LR ? int(threadIdx.x) % LR : int(threadIdx.x);
    const int64_t n = LR ? int64_t(blockIdx.x) * (256 / (LR ? LR : 1)) + threadIdx.x / (LR ? LR : 1) : int64_t(blockIdx.x);
    if (LR && n >= A.N) return;
    const int D = A.D;

    // over the row's lanes; `red` is free again when the next one starts (two barriers each)
    auto row_reduce = [&](auto op, uint32_t v) {
        using OP = decltype(op);
        if constexpr (LR != 0) {
            return lanes_reduce<OP, LR>(v);
        } else {
            v = lanes_reduce<OP, 64>(v);
            const int waves = int(blockDim.x) >> 6;
            if (waves == 1) return v;
            if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
            __syncthreads();
            // (sums in one order whatever the wavefront)
            uint32_t all = red[0];
            for (int w = 1; w < waves; ++w) all = OP::of(all, red[w]);
            __syncthreads();
            return all;
        }
    };

    float h[V][8];
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int j = (c * lanes + lane) * 8, left = D - j;
        if (left > 0) {
            load_chunk<T>(A.x, n * A.x_row + j, left, h[c]);
            if (A.residual) {
                float r[8];
                load_chunk<T>(A.residual, n * A.r_row + j, left, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[c][i] += r[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = 0.f;
        }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int j = (c * lanes + lane) * 8, left = D - j;
        if (A.residual && left > 0) store_chunk<T>(A.residual_out, n * A.ro_row + j, left, h[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(h[c][i], h[c][i], sum);
    }
    sum = __uint_as_float(row_reduce(OpAdd{}, __float_as_uint(sum)));
    float ms = sum / float(D) + A.eps;
    // Where the squares leave float32's range (|h| of 1.8e19 and more, or so small that they lose
    // bits against eps): h 2^-e and eps 2^-2e in their place, which gives the same y, with 2^e next
    // above the larger of max |h| and the root of eps. The row's lanes all go this way or none.
    if (!(ms >= 0x1p-100f && ms < INFINITY)) {
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) most = OpMax::of(most, magnitude(h[c][i]));
        most = row_reduce(OpMax{}, most);
        if (most < 0x7F800000u) {                        // (an infinity or a NaN stays as it is)
            const int eh = most ? __builtin_amdgcn_frexp_expf(__uint_as_float(most)) : -1000;
            const int ee = A.eps > 0.f ? (__builtin_amdgcn_frexp_expf(A.eps) + 1) >> 1 : -1000;
            const int e = most || A.eps > 0.f ? max(eh, ee) : 0;
            sum = 0.f;
#pragma unroll
            for (int c = 0; c < V; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    h[c][i] = __builtin_amdgcn_ldexpf(h[c][i], -e);
                    sum = __builtin_fmaf(h[c][i], h[c][i], sum);
                }
            sum = __uint_as_float(row_reduce(OpAdd{}, __float_as_uint(sum)));
            ms = sum / float(D) + __builtin_amdgcn_ldexpf(A.eps, -2 * e);
        }
    }
    // (a row of zeros without eps: any factor keeps its zeros, 0 * infinity would not)
    const float rstd = ms == 0.f ? 1.f : 1.f / sqrtf(ms);
    // rstd = pow2 * frac, frac in [1, 2): the row's z = h * pow2 * w is rounded once, y = z * frac,
    // and y / scale = z * 448 / max |z| has none of rstd's roundings
    const float pow2 = rstd != rstd ? rstd : __uint_as_float(__float_as_uint(rstd) & 0x7F800000u);
    const float frac = __uint_as_float((__float_as_uint(rstd) & 0x7FFFFFu) | 0x3F800000u);

    uint32_t top[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int j = (c * lanes + lane) * 8, left = D - j;
        float w[8];
        if (A.weight && left > 0) load_chunk<T>(A.weight, j, left, w);
        top[c] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[c][i] *= pow2;
            if (A.weight && left > 0) h[c][i] *= w[i];
            // (columns behind the row are 0 * pow2: NaN where the row's sum is)
            top[c] = OpMax::of(top[c], i < left ? magnitude(h[c][i]) : 0u);
        }
    }
    if (A.group == 0) {
        uint32_t all = top[0];
#pragma unroll
        for (int c = 1; c < V; ++c) all = OpMax::of(all, top[c]);
        all = row_reduce(OpMax{}, all);
#pragma unroll
        for (int c = 0; c < V; ++c) top[c] = all;
    } else {
#pragma unroll
        for (int c = 0; c < V; ++c) top[c] = lanes_reduce<OpMax, LR == 8 ? 8 : 16>(top[c]);
    }
    const int groups = A.group ? (D + 127) / 128 : 1;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const int j = (c * lanes + lane) * 8, left = D - j;
        if (left <= 0) continue;
        const float most = __uint_as_float(top[c]), scale = e4m3_scale(most * frac);
        const Factor by = codes_of(most, frac, scale);
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __builtin_fmaf(h[c][i], by.hi, h[c][i] * by.lo);
        u32x2 w;
        w[0] = e4m3_pack4(q[0], q[1], q[2], q[3]);
        w[1] = e4m3_pack4(q[4], q[5], q[6], q[7]);
        store_codes(A.codes + n * A.c_row + j, left, w);
        if (A.group ? (lane & 15) == 0 : c == 0 && lane == 0) A.scales[n * groups + (A.group ? j >> 7 : 0)] = scale;
    }
}

template <int T>
hipError_t norm_t(const NormArgs& a, hipStream_t s) {
    const int chunks = (a.D + 7) / 8;
    auto rows = [&](int per) { return unsigned((a.N + per - 1) / per); };
    auto threads = [&](int v) { return unsigned(((chunks + v - 1) / v + 63) / 64 * 64); };
    if (chunks <= 8) norm_kernel<T, 8, 1><<<rows(32), 256, 0, s>>>(a);
    else if (chunks <= 16) norm_kernel<T, 16, 1><<<rows(16), 256, 0, s>>>(a);
    else if (chunks <= 32) norm_kernel<T, 32, 1><<<rows(8), 256, 0, s>>>(a);
    else if (chunks <= 64) norm_kernel<T, 64, 1><<<rows(4), 256, 0, s>>>(a);
    else if (chunks <= 2048) norm_kernel<T, 0, 2><<<a.N, threads(2), 0, s>>>(a);
    else if (chunks <= 4096) norm_kernel<T, 0, 4><<<a.N, threads(4), 0, s>>>(a);
    else norm_kernel<T, 0, 8><<<a.N, threads(8), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    const int64_t size = a.dtype == WB_F32 ? 4 : 2, groups = a.group ? (a.D + a.group - 1) / a.group : 1;
    const int64_t most = kLaunchItems / 1024 * (a.D <= 512 ? 16 : 1);      // (64 lanes a row, or a workgroup)
    auto shifted = [](const void* p, int64_t bytes) { return p ? static_cast<const uint8_t*>(p) + bytes : nullptr; };
    for (int64_t n0 = 0; n0 < a.N; n0 += most) {
        NormArgs b = a;
        b.N = int(a.N - n0 < most ? a.N - n0 : most);
        b.x = shifted(a.x, n0 * a.x_row * size);
        b.residual = shifted(a.residual, n0 * a.r_row * size);
        b.residual_out = const_cast<uint8_t*>(shifted(a.residual_out, n0 * a.ro_row * size));
        b.codes = a.codes + n0 * a.c_row;
        b.scales = a.scales + n0 * groups;
        const hipError_t e = a.dtype == WB_BF16 ? norm_t<WB_BF16>(b, s) : a.dtype == WB_F16 ? norm_t<WB_F16>(b, s) : norm_t<WB_F32>(b, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace wb
