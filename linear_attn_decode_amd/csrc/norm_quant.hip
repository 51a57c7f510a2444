// Root-mean-square norm with the residual's addition and an e4m3 output (wbserve.h).
#include "serve_device.hpp"

namespace wb {
namespace {

template <int T>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if constexpr (T == WB_F32) return static_cast<const float*>(p)[i];
    else return Elem<T>::get(static_cast<const uint16_t*>(p)[i]);
}
template <int T>
__device__ __forceinline__ void store1(void* p, int64_t i, float x) {
    if constexpr (T == WB_F32) static_cast<float*>(p)[i] = x;
    else static_cast<uint16_t*>(p)[i] = Elem<T>::put(x);
}

// Any width, stride and alignment: a workgroup per row, one column a lane.
constexpr int kRowThreads = 256;

template <int T>
__global__ void __launch_bounds__(kRowThreads) norm_any_kernel(const NormArgs A) {
    __shared__ float red[kRowThreads / 64];
    const int tid = threadIdx.x, D = A.D;
    const int64_t n = blockIdx.x;
    auto h_at = [&](int j) {
        const float x = load1<T>(A.x, n * A.x_row + j);
        return A.residual ? x + load1<T>(A.residual, n * A.r_row + j) : x;
    };
    float sum = 0.f;
    for (int j = tid; j < D; j += kRowThreads) {
        const float h = h_at(j);
        sum = __builtin_fmaf(h, h, sum);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
    if ((tid & 63) == 0) red[tid >> 6] = sum;
    __syncthreads();
    sum = (red[0] + red[1]) + (red[2] + red[3]);
    const float rstd = 1.f / sqrtf(sum / float(D) + A.eps);
    auto y_at = [&](int j) { return h_at(j) * rstd * (A.weight ? load1<T>(A.weight, j) : 1.f); };

    const int group = A.group ? A.group : D, groups = (D + group - 1) / group;
    for (int g = 0; g < groups; ++g) {
        const int from = g * group, to = min(D, from + group);
        float top = 0.f;
        for (int j = from + tid; j < to; j += kRowThreads) top = max_nan(top, fabsf(y_at(j)));
#pragma unroll
        for (int d = 32; d; d >>= 1) top = max_nan(top, __shfl_xor(top, d, 64));
        __syncthreads();
        if ((tid & 63) == 0) red[tid >> 6] = top;
        __syncthreads();
        top = max_nan(max_nan(red[0], red[1]), max_nan(red[2], red[3]));
        const float scale = e4m3_scale(top), by = e4m3_divisor(scale);
        for (int j = from + tid; j < to; j += kRowThreads)
            A.codes[n * A.c_row + j] = uint8_t(e4m3_pack4(y_at(j) / by, 0.f, 0.f, 0.f));
        if (tid == 0) A.scales[n * groups + g] = scale;
    }
    // (last: the residual may be stored over the one that was read)
    if (A.residual) {
        __syncthreads();
        for (int j = tid; j < D; j += kRowThreads) store1<T>(A.residual_out, n * A.ro_row + j, h_at(j));
    }
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    if (a.N == 0) return hipSuccess;
    if (a.dtype == WB_BF16) norm_any_kernel<WB_BF16><<<a.N, kRowThreads, 0, s>>>(a);
    else if (a.dtype == WB_F16) norm_any_kernel<WB_F16><<<a.N, kRowThreads, 0, s>>>(a);
    else norm_any_kernel<WB_F32><<<a.N, kRowThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace wb
