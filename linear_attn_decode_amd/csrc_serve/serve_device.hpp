// Device helpers of the serving operators (gfx950, wave64): 16-bit and e4m3 conversions,
// lane reductions and scans.
#pragma once

#include "serve_kernels.hpp"
#include "wb_device.hpp"

namespace wb {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kE4M3Max = 448.0f;

// Element type T of the WB_* code: conversions of a 16-bit pattern and a pair of values
template <int T>
struct Elem;
template <>
struct Elem<WB_BF16> {
    static constexpr int size = 2;
    static __device__ __forceinline__ float get(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }
    static __device__ __forceinline__ uint16_t put(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
};
template <>
struct Elem<WB_F16> {
    static constexpr int size = 2;
    static __device__ __forceinline__ float get(uint16_t b) { return float(__builtin_bit_cast(_Float16, b)); }
    static __device__ __forceinline__ uint16_t put(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
};
template <>
struct Elem<WB_F32> {
    static constexpr int size = 4;
};

// Four e4m3 codes of four values already scaled into [-448, 448], to nearest with ties to
// the even code (NaN and values past the range give the NaN code)
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return uint32_t(w);
}

// The scale of a group whose largest magnitude is `top`, and what its quotients are taken
// with. A scale below the normal numbers would be rounded so coarsely that quotients pass
// 448: there it is the smallest normal number. A zero group divides by 1 (every code is 0).
__device__ __forceinline__ float e4m3_scale(float top) {
    const float s = top / kE4M3Max;
    return s < 0x1p-126f && top > 0.f ? 0x1p-126f : s;
}
__device__ __forceinline__ float e4m3_divisor(float scale) { return scale == 0.f ? 1.f : scale; }

// y / by for a divisor whose reciprocal (rcp = 1 / by) is taken once per group: the product
// corrected by its remainder, which is the quotient rounded to nearest but for rare ties.
// An infinite divisor gives NaN.
__device__ __forceinline__ float quotient(float y, float by, float rcp) {
    const float q = y * rcp;
    return __builtin_fmaf(__builtin_fmaf(-q, by, y), rcp, q);
}

// Magnitudes are compared as their bit patterns: for non-negative floats the order is the
// same, and a NaN is larger than everything, so that a maximum keeps it.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Reductions over 2^k neighbouring lanes (every lane gets the result): DPP inside rows of 16,
// lane swaps across them.
struct OpMax {
    static __device__ __forceinline__ uint32_t of(uint32_t a, uint32_t b) { return a > b ? a : b; }
};
struct OpAdd {
    static __device__ __forceinline__ uint32_t of(uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }
};
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false));
}
template <typename OP, int LANES>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t v) {
    static_assert(LANES == 8 || LANES == 16 || LANES == 32 || LANES == 64, "lanes of a reduction");
    v = OP::of(v, dpp_u32<0xB1>(v));       // quad_perm: xor 1
    v = OP::of(v, dpp_u32<0x4E>(v));       // quad_perm: xor 2
    v = OP::of(v, dpp_u32<0x141>(v));      // row_half_mirror: the other quad of 8
    if constexpr (LANES >= 16) v = OP::of(v, dpp_u32<0x140>(v));      // row_mirror: the other 8 of 16
    if constexpr (LANES >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = OP::of(p[0], p[1]);
    }
    if constexpr (LANES == 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = OP::of(p[0], p[1]);
    }
    return v;
}

// Lane swaps: v combined with the value the lane 32 / 16 apart holds
__device__ __forceinline__ float max_xor32(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float max_xor16(float v) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// Inclusive sum over the lanes of a wavefront (DPP: shifts inside rows of 16, then the rows' last lanes)
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t dpp_i64(int64_t v) {
    const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xF, false));
    const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(0, int(v >> 32), CTRL, ROWS, 0xF, false));
    return int64_t(uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
    v += dpp_i64<0x111, 0xF>(v);    // row_shr:1, 2, 4, 8
    v += dpp_i64<0x112, 0xF>(v);
    v += dpp_i64<0x114, 0xF>(v);
    v += dpp_i64<0x118, 0xF>(v);
    v += dpp_i64<0x142, 0xA>(v);    // row_bcast:15 into rows 1 and 3
    v += dpp_i64<0x143, 0xC>(v);    // row_bcast:31 into rows 2 and 3
    return v;
}

// a / b of non-negative numbers, in 32 bits where they fit (a 64-bit division is some 150
// dependent instructions)
__device__ __forceinline__ int64_t quotient64(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return int64_t(uint32_t(a) / uint32_t(b));
    return a / b;
}

__device__ __forceinline__ int64_t lane64(int64_t v, int lane) {
    return int64_t(uint64_t(uint32_t(__builtin_amdgcn_readlane(int(v), lane))) |
                   uint64_t(uint32_t(__builtin_amdgcn_readlane(int(v >> 32), lane))) << 32);
}

// 64 bits between workgroups of one launch, past the caches that the compute dies do not share
__device__ __forceinline__ void put_word(uint64_t* p, uint64_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get_word(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void stores_complete() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Whether this is the last of `count` workgroups to come here. The counter needs no clearing:
// it holds the call's tag above its 12 bits of count, whoever finds another tag there puts
// the call's with a count of 0 (one exchange; it fails only where another workgroup's has
// succeeded), and the last one takes the tag out again, so that a replay of a captured call,
// which has the same tag, starts over. Nothing waits here.
constexpr int kCountBits = 12;
__device__ __forceinline__ bool last_to_arrive(uint64_t* c, uint64_t tag, int count) {
    uint64_t v = __hip_atomic_load(c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (v >> kCountBits != tag)
        __hip_atomic_compare_exchange_strong(c, &v, tag << kCountBits, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
    v = __hip_atomic_fetch_add(c, uint64_t(1), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const bool last = int(v & ((1u << kCountBits) - 1)) + 1 == count;
    if (last) __hip_atomic_store(c, uint64_t(0), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return last;
}

}  // namespace wb
