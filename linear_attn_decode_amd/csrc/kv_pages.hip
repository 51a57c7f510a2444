// Page planning and cache writes of the paged key-value cache (wbserve.h).
#include "serve_device.hpp"

namespace wb {
namespace {

// ---------------------------------------------------------------------------
// Planning is two sums over the requests (pages taken, new tokens) and a scatter. One
// workgroup takes the sums for any number of requests: it first decides whether the whole
// plan can be carried out (nothing has been written by then, so an output may be its
// input), then writes it. Up to kPlanSlots slots it also writes the slots, so that a
// decode step's plan is one launch; more are written by a second launch of many
// workgroups, which takes the pages before each request from `work`.
constexpr int kPlanRows = 1024;        // requests whose sums are kept in LDS
constexpr int64_t kPlanSlots = 4096;
constexpr int kFillPerThread = 4, kFillThreads = 256;

struct PlanShared {
    int starts[kPlanRows + 1];
    int first[kPlanRows];
    int old[kPlanRows];
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

// Slot of new token i of request r, and the table entry where it begins a new page.
__device__ __forceinline__ int64_t place(const PlanArgs& A, int n_free, int r, int i, int start, int old, int first) {
    const int64_t pos = int64_t(old) + (i - start);
    const int j = int(pos >> A.page_log2), have = pages_of(old, A.page_log2);
    const size_t at = size_t(r) * A.width + j;
    int page;
    if (j >= have) {
        page = A.free_pages[n_free - 1 - first - (j - have)];
        // (a new page is entered at its first token: those held end at or before it)
        if ((pos & ((int64_t(1) << A.page_log2) - 1)) == 0) A.table[at] = page;
    } else {
        page = A.table[at];
    }
    return (int64_t(page) << A.page_log2) + (pos & ((int64_t(1) << A.page_log2) - 1));
}

template <int NT>
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* lds) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    int64_t s = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) s += lds[w];
    return s;
}

// Exclusive sum over the workgroup's threads; *total their sum.
template <int NT>
__device__ __forceinline__ int block_scan(int v, int* lds, int* total) {
    const int inc = wave_scan(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = inc;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        const int x = lds[w];
        if (w < int(threadIdx.x >> 6)) before += x;
        sum += x;
    }
    *total = sum;
    return before + inc - v;
}

template <int NT, bool SLOTS>
__global__ void __launch_bounds__(NT) plan_kernel(const PlanArgs A) {
    __shared__ PlanShared sh;
    __shared__ int64_t red[NT / 64];
    __shared__ int scan[NT / 64];
    const int tid = threadIdx.x, R = A.R;
    const int n_free = *A.n_free;

    int64_t tokens = 0, pages = 0;
    int bad = 0;                                     // bit 0: status 1, bit 1: status 2
    for (int r = tid; r < R; r += NT) {
        const int old = A.lens[r], more = A.more[r];
        if (old < 0 || more < 0) {
            bad |= 1;
            continue;
        }
        const int want = pages_of(int64_t(old) + more, A.page_log2);
        if (want > A.width) bad |= 2;
        tokens += more;
        pages += want - pages_of(old, A.page_log2);
    }
    if (n_free < 0 || n_free > A.free_size) bad |= 1;
    const int any1 = __syncthreads_or(bad & 1), any2 = __syncthreads_or(bad & 2);
    tokens = block_sum<NT>(tokens, red);
    pages = block_sum<NT>(pages, red);
    const int status = any1 ? 1 : any2 ? 2 : tokens > A.n_slots ? 3 : pages > n_free ? 4 : 0;

    int before_tok = 0, before_pages = 0;
    for (int base = 0; base < R; base += NT) {
        const int r = base + tid;
        const int old = r < R ? A.lens[r] : 0, more = r < R && !status ? A.more[r] : 0;
        const int take = status ? 0 : pages_of(int64_t(old) + more, A.page_log2) - pages_of(old, A.page_log2);
        int sum_tok, sum_pages;
        const int start = before_tok + block_scan<NT>(more, scan, &sum_tok);
        const int first = before_pages + block_scan<NT>(take, scan, &sum_pages);
        before_tok += sum_tok;
        before_pages += sum_pages;
        if (r < R) {
            A.starts[r] = start;
            A.lens_out[r] = old + more;
            if constexpr (SLOTS) {
                sh.starts[r] = start;
                sh.first[r] = first;
                sh.old[r] = old;
            } else {
                A.work[r] = first;
            }
        }
    }
    if (tid == 0) {
        A.starts[R] = before_tok;
        *A.n_free_out = n_free - before_pages;
        *A.status = status;
    }
    if constexpr (SLOTS) {
        __syncthreads();
        for (int i = tid; i < A.n_slots; i += NT) {
            int64_t slot = -1;
            if (i < before_tok) {
                const int r = row_of(sh.starts, R, i);
                slot = place(A, n_free, r, i, sh.starts[r], sh.old[r], sh.first[r]);
            }
            A.slots[i] = slot;
        }
    }
}

__global__ void __launch_bounds__(kFillThreads) plan_slots_kernel(const PlanArgs A) {
    const int64_t i0 = (int64_t(blockIdx.x) * kFillThreads + threadIdx.x) * kFillPerThread;
    if (i0 >= A.n_slots) return;
    const int total = A.starts[A.R];
    // (n_free_out may be n_free: the stack's height before the pages were taken)
    const int last = A.R - 1;
    int64_t slot[kFillPerThread];
    int r = total ? row_of(A.starts, A.R, int(i0 < total ? i0 : total - 1)) : last;
    int n_free = 0;
    if (total) {
        const int more = A.starts[last + 1] - A.starts[last], len = A.lens_out[last];
        n_free = *A.n_free_out + A.work[last] + pages_of(len, A.page_log2) - pages_of(len - more, A.page_log2);
    }
#pragma unroll
    for (int x = 0; x < kFillPerThread; ++x) {
        const int64_t i = i0 + x;
        slot[x] = -1;
        if (i < total) {
            while (A.starts[r + 1] <= i) ++r;
            const int start = A.starts[r], old = A.lens_out[r] - (A.starts[r + 1] - start);
            slot[x] = place(A, n_free, r, int(i), start, old, A.work[r]);
        }
    }
    if (i0 + kFillPerThread <= A.n_slots) {
        int64_t* out = A.slots + i0;
#pragma unroll
        for (int x = 0; x < kFillPerThread; x += 2)
            *reinterpret_cast<longlong2*>(out + x) = make_longlong2(slot[x], slot[x + 1]);
    } else {
        for (int x = 0; i0 + x < A.n_slots; ++x) A.slots[i0 + x] = slot[x];
    }
}

constexpr int kReleaseThreads = 1024;
__global__ void __launch_bounds__(kReleaseThreads) release_kernel(const ReleaseArgs A) {
    constexpr int NT = kReleaseThreads;
    __shared__ int64_t red[NT / 64];
    __shared__ int scan[NT / 64];
    __shared__ int at[NT], count[NT];
    const int tid = threadIdx.x, R = A.R;
    const int n_free = *A.n_free;
    int64_t pages = 0;
    int bad = n_free < 0 || n_free > A.free_size;
    for (int r = tid; r < R; r += NT) {
        const int len = A.lens[r];
        if (len < 0) bad |= 1;
        else if (A.ended[r]) {
            const int n = pages_of(len, A.page_log2);
            if (n > A.width) bad |= 2;
            pages += n;
        }
    }
    const int any1 = __syncthreads_or(bad & 1), any2 = __syncthreads_or(bad & 2);
    pages = block_sum<NT>(pages, red);
    const int status = any1 ? 1 : any2 ? 2 : n_free + pages > A.free_size ? 4 : 0;
    if (tid == 0) *A.status = status;
    if (status) return;
    int before = n_free;
    for (int base = 0; base < R; base += NT) {
        const int r = base + tid;
        const int n = r < R && A.ended[r] ? pages_of(A.lens[r], A.page_log2) : 0;
        int sum;
        const int mine = before + block_scan<NT>(n, scan, &sum);
        before += sum;
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
    if (tid == 0) *A.n_free = before;
}

// ---------------------------------------------------------------------------
// Cache writes. A lane holds 8 values of a vector, D / 8 neighbouring lanes the vector;
// lanes of one wavefront take consecutive vectors of one token's heads, so rows are read
// in order. Bound by HBM: every input value is read once and every stored byte written
// once; the vector's maximum is taken by lane exchanges inside its D / 8 lanes.
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

template <int DST, int SRC, int D>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs A) {
    constexpr int L = D / 8;                          // lanes of a vector
    const int H = A.c.H;
    const int64_t vec = (int64_t(blockIdx.x) * 256 + threadIdx.x) / L;
    if (vec >= int64_t(A.N) * H) return;
    const int lane = threadIdx.x % L;
    const int64_t i = vec / H;
    const int h = int(vec - i * H);
    const bool is_v = blockIdx.y;
    const int64_t slot = A.slots[i];
    if (slot < 0 || slot >= (A.c.pages << A.page_log2)) return;
    const int64_t page = slot >> A.page_log2, off = slot & ((1 << A.page_log2) - 1);
    const int64_t row = ((page * H + h) << A.page_log2) + off;
    const void* src = is_v ? A.v : A.k;
    void* dst = is_v ? A.c.v : A.c.k;
    const int64_t from = i * (is_v ? A.v_row : A.k_row) + int64_t(h) * D + lane * 8;
    if constexpr (DST == SRC) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(src) + from);
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(dst) + row * D + lane * 8) = w;
    } else {
        float x[8];
        load8<SRC>(src, from, x);
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
            *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(dst) + row * D + lane * 8) = w;
            if (lane == 0) (is_v ? A.c.v_scale : A.c.k_scale)[row] = scale;
        } else {
            u32x4 w;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = uint32_t(Elem<DST>::put(x[2 * j])) | (uint32_t(Elem<DST>::put(x[2 * j + 1])) << 16);
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(dst) + row * D + lane * 8) = w;
        }
    }
}

template <int DST, int SRC>
hipError_t append_d(const AppendArgs& a, hipStream_t s) {
    const int64_t lanes = int64_t(a.N) * a.c.H * (a.c.D / 8);
    const dim3 grid(unsigned((lanes + 255) / 256), 2);
    switch (a.c.D) {
        case 64: append_kernel<DST, SRC, 64><<<grid, 256, 0, s>>>(a); break;
        case 128: append_kernel<DST, SRC, 128><<<grid, 256, 0, s>>>(a); break;
        default: append_kernel<DST, SRC, 256><<<grid, 256, 0, s>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace

bool plan_in_one_launch(int R, int64_t n_slots) { return R <= kPlanRows && n_slots <= kPlanSlots; }

hipError_t launch_plan(const PlanArgs& a, hipStream_t s) {
    if (plan_in_one_launch(a.R, a.n_slots)) {
        if (a.R <= 256 && a.n_slots <= 1024) plan_kernel<256, true><<<1, 256, 0, s>>>(a);
        else plan_kernel<1024, true><<<1, 1024, 0, s>>>(a);
        return hipGetLastError();
    }
    plan_kernel<1024, false><<<1, 1024, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.n_slots == 0) return e;
    constexpr int64_t per = kFillThreads * kFillPerThread;
    plan_slots_kernel<<<unsigned((a.n_slots + per - 1) / per), kFillThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_release(const ReleaseArgs& a, hipStream_t s) {
    release_kernel<<<1, kReleaseThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_append(const AppendArgs& a, hipStream_t s) {
    if (a.c.dtype == WB_E4M3) {
        if (a.src == WB_BF16) return append_d<WB_E4M3, WB_BF16>(a, s);
        if (a.src == WB_F16) return append_d<WB_E4M3, WB_F16>(a, s);
        return append_d<WB_E4M3, WB_F32>(a, s);
    }
    if (a.c.dtype == WB_BF16) return a.src == WB_F32 ? append_d<WB_BF16, WB_F32>(a, s) : append_d<WB_BF16, WB_BF16>(a, s);
    return a.src == WB_F32 ? append_d<WB_F16, WB_F32>(a, s) : append_d<WB_F16, WB_F16>(a, s);
}

}  // namespace wb
