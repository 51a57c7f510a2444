// Page planning and cache writes of the paged key-value cache (wbserve.h).
#include "serve_device.hpp"

namespace wb {
namespace {

// ---------------------------------------------------------------------------
// Planning is two sums over the requests (pages taken, new tokens) and a scatter; it is bound
// by latency, and by the 8 bytes a slot for plans of whole prompts. Three forms:
//   * Few slots (a decode step): one workgroup takes the sums and writes everything. It first
//     decides whether the whole plan can be carried out, so an output may be its input.
//   * Many slots of up to kPlanRows requests, outputs apart from inputs: every workgroup takes
//     the sums for itself (1.5 us, while one more launch costs the host 3.5 us and the GPU 5)
//     and writes its share of the slots; the first also writes the rest.
//   * Otherwise one workgroup takes the sums, which may be in place, and a second launch of many
//     workgroups writes the slots, with the pages before each request in `work`.
// Measured for 256 requests and 700 419 new tokens, in a graph: 7.3 us in the second form, 13.1
// us in the third (kernels of 4.9 and 9.7 us in a trace, 8.2 of the second form).
constexpr int kPlanRows = 1024;        // requests whose sums are kept in LDS
constexpr int64_t kPlanSlots = 4096;
constexpr int kFillPerThread = 8, kFillThreads = 256;

struct PlanShared {
    int starts[kPlanRows + 1];
    int first[kPlanRows];
    int old[kPlanRows], more[kPlanRows];
};

__device__ __forceinline__ int pages_of(int64_t tokens, int log2) {
    return int((tokens + (int64_t(1) << log2) - 1) >> log2);
}

// Last r in [0, n) with starts[r] <= i (starts ascending, starts[0] <= i): requests without
// new tokens share their start with the next one, which this passes on to.
__device__ __forceinline__ int row_of(const int* starts, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Page j of request r, which holds its token at `pos`: one of those taken, entered into the
// table at its first token (those held end at or before it), or one the request held.
__device__ __forceinline__ int page_for(const PlanArgs& A, int n_free, int r, int64_t pos, int old, int first) {
    const int j = int(pos >> A.page_log2), have = pages_of(old, A.page_log2);
    const size_t at = size_t(r) * A.width + j;
    if (j < have) return A.table[at];
    const int page = A.free_pages[n_free - 1 - first - (j - have)];
    if ((pos & ((int64_t(1) << A.page_log2) - 1)) == 0) A.table[at] = page;
    return page;
}

// kFillPerThread slots from i0: starts, first (pages before) and old length of the requests by
// the functions given; new tokens end at `total`. A page is looked up once for its slots.
template <typename START, typename FIRST, typename OLD>
__device__ __forceinline__ void fill_slots(const PlanArgs& A, int n_free, int64_t i0, int total, int r, START start,
                                           FIRST first, OLD old, int64_t slot[kFillPerThread]) {
    const int mask = (1 << A.page_log2) - 1;
    int64_t pos = 0, page = 0;
    int left = 0;                                    // new tokens of request r from i on
    bool look = true;
#pragma unroll
    for (int x = 0; x < kFillPerThread; ++x) {
        const int64_t i = i0 + x;
        slot[x] = -1;
        if (i >= total) continue;
        if (x == 0 || left == 0) {
            while (start(r + 1) <= i) ++r;
            left = int(start(r + 1) - i);
            pos = int64_t(old(r)) + (i - start(r));
            look = true;
        }
        if (look || (pos & mask) == 0) page = page_for(A, n_free, r, pos, old(r), first(r));
        look = false;
        slot[x] = (page << A.page_log2) + (pos & mask);
        ++pos;
        --left;
    }
}

// Over a workgroup of NT threads: exclusive sums of two counts and the bits any thread set,
// behind what `sum` holds already (all threads agree on it).
struct Sums {
    int64_t a, b;
    int bits;
};
template <int NT>
struct ScanLds {
    int64_t a[NT / 64], b[NT / 64];
    int bits[NT / 64];
};
template <int NT>
__device__ __forceinline__ Sums block_scan(int64_t a, int64_t b, int bits, Sums& sum, ScanLds<NT>& lds) {
    const int wave = threadIdx.x >> 6;
    const int64_t ia = wave_scan(a), ib = wave_scan(b);
    const int any = (__any(bits & 1) ? 1 : 0) | (__any(bits & 2) ? 2 : 0);
    __syncthreads();                                 // (the last scan's have been read)
    if ((threadIdx.x & 63) == 63) {
        lds.a[wave] = ia;
        lds.b[wave] = ib;
        lds.bits[wave] = any;
    }
    __syncthreads();
    Sums before = sum;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        if (w < wave) {
            before.a += lds.a[w];
            before.b += lds.b[w];
        }
        sum.a += lds.a[w];
        sum.b += lds.b[w];
        sum.bits |= lds.bits[w];
    }
    before.a += ia - a;
    before.b += ib - b;
    return before;
}

// A thread's slots in a row, 16 bytes at a time where they are all inside.
__device__ __forceinline__ void store_slots(const PlanArgs& A, int64_t i0, const int64_t slot[kFillPerThread]) {
    if (i0 + kFillPerThread <= A.n_slots) {
        int64_t* out = A.slots + i0;
#pragma unroll
        for (int x = 0; x < kFillPerThread; x += 2)
            *reinterpret_cast<longlong2*>(out + x) = make_longlong2(slot[x], slot[x + 1]);
    } else {
#pragma unroll
        for (int x = 0; x < kFillPerThread; ++x)
            if (i0 + x < A.n_slots) A.slots[i0 + x] = slot[x];
    }
}

enum PlanForm { kPlanOne, kPlanSpread, kPlanSums };     // one workgroup; one launch; sums for the second launch

template <int NT, PlanForm FORM>
__global__ void __launch_bounds__(NT) plan_kernel(const PlanArgs A) {
    constexpr bool kRows = FORM != kPlanSums;        // the sums stay in LDS
    __shared__ PlanShared sh;
    __shared__ ScanLds<NT> lds;
    const int tid = threadIdx.x, R = A.R;
    const bool writer = FORM != kPlanSpread || blockIdx.x == 0;
    const int n_free = *A.n_free;

    // new tokens and pages taken; bits: status 1, status 2. A request that is out of range
    // counts nothing (the plan is not carried out), so that the sums cannot overflow.
    Sums sum{0, 0, n_free < 0 || n_free > A.free_size ? 1 : 0};
    for (int base = 0; base < R; base += NT) {
        const int r = base + tid;
        int old = r < R ? A.lens[r] : 0, more = r < R ? A.more[r] : 0, bits = 0;
        if (old < 0 || more < 0) bits = 1;
        else if (pages_of(int64_t(old) + more, A.page_log2) > A.width) bits = 2;
        const int take = bits ? 0 : pages_of(int64_t(old) + more, A.page_log2) - pages_of(old, A.page_log2);
        const Sums at = block_scan<NT>(bits ? 0 : more, take, bits, sum, lds);
        if (kRows && r < R) {
            sh.starts[r] = int(at.a);
            sh.first[r] = int(at.b);
            sh.old[r] = old;
            sh.more[r] = more;
        }
    }
    const int status = sum.bits & 1 ? 1 : sum.bits ? 2 : sum.a > A.n_slots ? 3 : sum.b > n_free ? 4 : 0;
    const int before_tok = status ? 0 : int(sum.a), before_pages = status ? 0 : int(sum.b);
    if constexpr (kRows) {
        if (writer)
            for (int r = tid; r < R; r += NT) {      // (a thread's own rows)
                A.starts[r] = status ? 0 : sh.starts[r];
                A.lens_out[r] = sh.old[r] + (status ? 0 : sh.more[r]);
            }
    } else {
        Sums again{0, 0, 0};
        for (int base = 0; base < R; base += NT) {
            const int r = base + tid;
            const int old = r < R ? A.lens[r] : 0, more = r < R && !status ? A.more[r] : 0;
            const int take = status ? 0 : pages_of(int64_t(old) + more, A.page_log2) - pages_of(old, A.page_log2);
            const Sums at = block_scan<NT>(more, take, 0, again, lds);
            if (r < R) {
                A.starts[r] = int(at.a);
                A.lens_out[r] = old + more;
                A.work[r] = int(at.b);
            }
        }
    }
    if (tid == 0 && writer) {
        A.starts[R] = before_tok;
        *A.n_free_out = n_free - before_pages;
        *A.status = status;
    }
    if constexpr (FORM == kPlanOne) {
        __syncthreads();
        for (int i = tid; i < A.n_slots; i += NT) {
            int64_t slot = -1;
            if (i < before_tok) {
                const int r = row_of(sh.starts, R, i);
                const int64_t pos = int64_t(sh.old[r]) + (i - sh.starts[r]);
                slot = (int64_t(page_for(A, n_free, r, pos, sh.old[r], sh.first[r])) << A.page_log2) +
                       (pos & ((int64_t(1) << A.page_log2) - 1));
            }
            A.slots[i] = slot;
        }
    } else if constexpr (FORM == kPlanSpread) {
        if (tid == 0) sh.starts[R] = before_tok;
        __syncthreads();
        const int64_t i0 = (int64_t(blockIdx.x) * NT + tid) * kFillPerThread;
        if (i0 >= A.n_slots) return;
        int64_t slot[kFillPerThread];
        const int r = before_tok ? row_of(sh.starts, R, int(i0 < before_tok ? i0 : before_tok - 1)) : 0;
        fill_slots(A, n_free, i0, before_tok, r, [&](int x) { return sh.starts[x]; }, [&](int x) { return sh.first[x]; },
                   [&](int x) { return sh.old[x]; }, slot);
        store_slots(A, i0, slot);
    }
}

__global__ void __launch_bounds__(kFillThreads) plan_slots_kernel(const PlanArgs A) {
    const int64_t i0 = (int64_t(blockIdx.x) * kFillThreads + threadIdx.x) * kFillPerThread;
    if (i0 >= A.n_slots) return;
    const int total = A.starts[A.R];
    // (n_free_out may be n_free: the stack's height before the pages were taken)
    const int last = A.R - 1;
    int64_t slot[kFillPerThread];
    const int r = total ? row_of(A.starts, A.R, int(i0 < total ? i0 : total - 1)) : last;
    int n_free = 0;
    if (total) {
        const int more = A.starts[last + 1] - A.starts[last], len = A.lens_out[last];
        n_free = *A.n_free_out + A.work[last] + pages_of(len, A.page_log2) - pages_of(len - more, A.page_log2);
    }
    fill_slots(A, n_free, i0, total, r, [&](int x) { return A.starts[x]; }, [&](int x) { return A.work[x]; },
               [&](int x) { return A.lens_out[x] - (A.starts[x + 1] - A.starts[x]); }, slot);
    store_slots(A, i0, slot);
}

constexpr int kReleaseThreads = 1024;
__global__ void __launch_bounds__(kReleaseThreads) release_kernel(const ReleaseArgs A) {
    constexpr int NT = kReleaseThreads;
    __shared__ ScanLds<NT> lds;
    __shared__ int at[NT], count[NT];
    const int tid = threadIdx.x, R = A.R;
    const int n_free = *A.n_free;
    auto pages_in = [&](int r) { return r < R && A.ended[r] && A.lens[r] > 0 ? pages_of(A.lens[r], A.page_log2) : 0; };
    Sums sum{0, 0, n_free < 0 || n_free > A.free_size ? 1 : 0};
    for (int base = 0; base < R; base += NT) {
        const int n = pages_in(base + tid);
        const int bits = base + tid < R && A.lens[base + tid] < 0 ? 1 : n > A.width ? 2 : 0;
        block_scan<NT>(n, 0, bits, sum, lds);
    }
    const int status = sum.bits & 1 ? 1 : sum.bits ? 2 : n_free + sum.a > A.free_size ? 4 : 0;
    if (tid == 0) *A.status = status;
    if (status) return;
    Sums again{n_free, 0, 0};
    for (int base = 0; base < R; base += NT) {
        const int r = base + tid, n = pages_in(r);
        const int mine = int(block_scan<NT>(n, 0, 0, again, lds).a);
        at[tid] = mine;
        count[tid] = n;
        if (r < R && A.ended[r]) A.lens[r] = 0;
        __syncthreads();
        // a wavefront per request, a lane per page
        for (int x = tid >> 6; x < NT && base + x < R; x += NT / 64)
            for (int j = tid & 63; j < count[x]; j += 64)
                A.free_pages[at[x] + j] = A.table[size_t(base + x) * A.width + j];
        __syncthreads();
    }
    if (tid == 0) *A.n_free = int(again.a);
}

// ---------------------------------------------------------------------------
// Cache writes. A lane holds 8 values of a key and of the value beside it, D / 8 neighbouring
// lanes the vectors; lanes of one wavefront take consecutive vectors of one token's heads, so
// rows are read in order. Bound by HBM: every input value is read once and every stored byte
// written once, past the caches (what a decode step reads back of it is one token a request);
// the vector's maximum is taken by lane exchanges inside its D / 8 lanes. 65536 tokens of 8
// heads of 128 columns into an e4m3 cache: 77.6 us, 5.25 TB/s (80.8 us with ordinary stores,
// 92.4 us with keys and values in workgroups of their own; a copy of 4 GiB runs at 4.7 TB/s).
template <int SRC>
__device__ __forceinline__ void load8(const void* p, int64_t at, float x[8]) {
    if constexpr (SRC == WB_F32) {
        const f32x4* s = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
        const f32x4 a = s[0], b = s[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = a[i];
            x[4 + i] = b[i];
        }
    } else {
        const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = Elem<SRC>::get(uint16_t(w[i]));
            x[2 * i + 1] = Elem<SRC>::get(uint16_t(w[i] >> 16));
        }
    }
}

// One vector's 8 values of this lane, stored as DST at `row` of a cache.
template <int DST, int SRC, int D>
__device__ __forceinline__ void store_vector(float x[8], void* dst, float* scales, int64_t row, int lane) {
    constexpr int L = D / 8;
    if constexpr (DST == WB_E4M3) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = OpMax::of(top, magnitude(x[j]));
        const float scale = e4m3_scale(__uint_as_float(lanes_reduce<OpMax, L>(top))), by = e4m3_divisor(scale);
        const float rcp = __builtin_amdgcn_rcpf(by);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = quotient(x[j], by, rcp);
        u32x2 w;
        w[0] = e4m3_pack4(x[0], x[1], x[2], x[3]);
        w[1] = e4m3_pack4(x[4], x[5], x[6], x[7]);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(static_cast<uint8_t*>(dst) + row * D + lane * 8));
        if (lane == 0) scales[row] = scale;
    } else {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = uint32_t(Elem<DST>::put(x[2 * j])) | (uint32_t(Elem<DST>::put(x[2 * j + 1])) << 16);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(dst) + row * D + lane * 8));
    }
}

template <int DST, int SRC, int D>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs A) {
    constexpr int L = D / 8;                          // lanes of a vector
    const uint32_t H = uint32_t(A.c.H), vec = blockIdx.x * (256 / L) + threadIdx.x / L;
    if (vec >= uint32_t(A.N) * H) return;
    const int lane = threadIdx.x % L;
    const uint32_t i = vec / H, h = vec - i * H;
    const int64_t slot = A.slots[i];
    if (slot < 0 || slot >= (A.c.pages << A.page_log2)) return;
    const int64_t page = slot >> A.page_log2, off = slot & ((1 << A.page_log2) - 1);
    const int64_t row = ((page * H + h) << A.page_log2) + off;
    const int64_t col = int64_t(h) * D + lane * 8;
    const int64_t k_at = i * A.k_row + col, v_at = i * A.v_row + col;
    if constexpr (DST == SRC) {
        const u32x4 k = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(A.k) + k_at);
        const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(A.v) + v_at);
        const int64_t to = row * D + lane * 8;
        __builtin_nontemporal_store(k, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(A.c.k) + to));
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(A.c.v) + to));
    } else {
        float k[8], v[8];
        load8<SRC>(A.k, k_at, k);
        load8<SRC>(A.v, v_at, v);
        store_vector<DST, SRC, D>(k, A.c.k, A.c.k_scale, row, lane);
        store_vector<DST, SRC, D>(v, A.c.v, A.c.v_scale, row, lane);
    }
}

template <int DST, int SRC>
hipError_t append_d(const AppendArgs& a, hipStream_t s) {
    const int64_t vectors = int64_t(a.N) * a.c.H, per = 256 / (a.c.D / 8);
    const unsigned grid = unsigned((vectors + per - 1) / per);
    switch (a.c.D) {
        case 64: append_kernel<DST, SRC, 64><<<grid, 256, 0, s>>>(a); break;
        case 128: append_kernel<DST, SRC, 128><<<grid, 256, 0, s>>>(a); break;
        default: append_kernel<DST, SRC, 256><<<grid, 256, 0, s>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace

int plan_work(int R, int64_t n_slots, bool in_place) {
    return R <= kPlanRows && (n_slots <= kPlanSlots || !in_place) ? 0 : R;
}

hipError_t launch_plan(const PlanArgs& a, hipStream_t s) {
    const bool in_place = a.lens_out == a.lens || a.n_free_out == a.n_free;
    constexpr int64_t per = kFillThreads * kFillPerThread;
    const unsigned fill = unsigned((a.n_slots + per - 1) / per);
    if (plan_work(a.R, a.n_slots, in_place) == 0) {
        if (a.R <= 256 && a.n_slots <= 1024) plan_kernel<256, kPlanOne><<<1, 256, 0, s>>>(a);
        else if (a.n_slots <= kPlanSlots) plan_kernel<1024, kPlanOne><<<1, 1024, 0, s>>>(a);
        else plan_kernel<kFillThreads, kPlanSpread><<<fill, kFillThreads, 0, s>>>(a);
        return hipGetLastError();
    }
    plan_kernel<1024, kPlanSums><<<1, 1024, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.n_slots == 0) return e;
    plan_slots_kernel<<<fill, kFillThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_release(const ReleaseArgs& a, hipStream_t s) {
    release_kernel<<<1, kReleaseThreads, 0, s>>>(a);
    return hipGetLastError();
}

static hipError_t append(const AppendArgs& a, hipStream_t s) {
    if (a.c.dtype == WB_E4M3) {
        if (a.src == WB_BF16) return append_d<WB_E4M3, WB_BF16>(a, s);
        if (a.src == WB_F16) return append_d<WB_E4M3, WB_F16>(a, s);
        return append_d<WB_E4M3, WB_F32>(a, s);
    }
    if (a.c.dtype == WB_BF16) return a.src == WB_F32 ? append_d<WB_BF16, WB_F32>(a, s) : append_d<WB_BF16, WB_BF16>(a, s);
    return a.src == WB_F32 ? append_d<WB_F16, WB_F32>(a, s) : append_d<WB_F16, WB_F16>(a, s);
}

hipError_t launch_append(const AppendArgs& a, hipStream_t s) {
    const int64_t size = a.src == WB_F32 ? 4 : 2, most = kLaunchItems / (int64_t(a.c.H) * (a.c.D / 8));
    for (int64_t i0 = 0; i0 < a.N; i0 += most) {
        AppendArgs b = a;
        b.N = int(a.N - i0 < most ? a.N - i0 : most);
        b.k = static_cast<const uint8_t*>(a.k) + i0 * a.k_row * size;
        b.v = static_cast<const uint8_t*>(a.v) + i0 * a.v_row * size;
        b.slots = a.slots + i0;
        const hipError_t e = append(b, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace wb
