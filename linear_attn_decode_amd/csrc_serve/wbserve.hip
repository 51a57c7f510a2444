// Host side of the serving operators' C ABI (include/wbserve.h): argument checks and
// dispatch. No device memory is allocated, and nothing of a call is kept for the next.
#include <time.h>
#include <unistd.h>

#include <atomic>

#include "serve_kernels.hpp"

namespace {

constexpr int kMaxRequests = 65536, kMaxQueryHeads = 4096, kMaxColumns = 65536;
constexpr int64_t kMaxTokens = int64_t(1) << 30;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? WB_OK : WB_ELAUNCH; }
int element_size(int t) { return t == WB_F32 ? 4 : t == WB_E4M3 ? 1 : 2; }

// log2 of a page size that is built, or -1
int page_log2(int page) {
    if (page < 8 || page > 4096 || (page & (page - 1))) return -1;
    return __builtin_ctz(unsigned(page));
}

int check_cache(const wb_kv_cache* c) {
    if (!c || !c->k || !c->v || c->pages < 1 || c->H < 1) return WB_EINVAL;
    if (c->dtype != WB_BF16 && c->dtype != WB_F16 && c->dtype != WB_E4M3) return WB_EINVAL;
    const bool scaled = c->dtype == WB_E4M3;
    if ((c->k_scale != nullptr) != scaled || (c->v_scale != nullptr) != scaled) return WB_EINVAL;
    if (page_log2(c->page) < 0 || (c->D != 64 && c->D != 128 && c->D != 256)) return WB_EUNSUPPORTED;
    if (c->pages > (int64_t(0x7FFFFFFF) >> page_log2(c->page)) || c->H > kMaxQueryHeads) return WB_EUNSUPPORTED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)) return WB_EALIGN;
    return WB_OK;
}

int check_table(int R, int width, int page) {
    if (R < 1 || width < 1) return WB_EINVAL;
    const int log2 = page_log2(page);
    if (log2 < 0 || R > kMaxRequests) return WB_EUNSUPPORTED;
    if (int64_t(width) > (kMaxTokens >> log2) || int64_t(R) * width > 0x7FFFFFFF) return WB_EUNSUPPORTED;
    return WB_OK;
}

// what kv_attend_work and kv_attend both check
int check_attend(const wb_kv_cache* c, int R, int Hq, int width) {
    int v = check_cache(c);
    if (v) return v;
    v = check_table(R, width, c->page);
    if (v) return v;
    if (Hq < 1 || Hq % c->H) return WB_EINVAL;
    return Hq > kMaxQueryHeads ? WB_EUNSUPPORTED : WB_OK;
}

size_t work_bytes_of(const wb::AttendPlan& p) {
    return p.part_o_bytes + p.part_ml_bytes + p.spans_bytes + p.arrivals_bytes;
}

// A call's tag, 52 bits: successive numbers from a start of the process's own, scrambled
// (SplitMix64's finaliser; Steele, Lea, Flood, OOPSLA 2014), so that whatever the workspace
// held before is the call's own tag with probability 2^-52.
uint64_t next_tag() {
    static std::atomic<uint64_t> next{[] {
        timespec t{};
        clock_gettime(CLOCK_REALTIME, &t);
        return uint64_t(t.tv_sec) * 1000000007u + uint64_t(t.tv_nsec) + (uint64_t(getpid()) << 40);
    }()};
    for (;;) {
        uint64_t z = next.fetch_add(1, std::memory_order_relaxed) * 0x9E3779B97F4A7C15ull;
        z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
        z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
        z = (z ^ (z >> 31)) >> 12;
        if (z) return z;
    }
}

}  // namespace

extern "C" {

int kv_plan_work(int R, int64_t n_slots, int in_place) { return wb::plan_work(R, n_slots, in_place != 0); }

int kv_plan_pages(const int32_t* lens, const int32_t* more, int R, int32_t* table, int width, const int32_t* free_pages,
                  int free_size, const int32_t* n_free, int page, int64_t* slots, int64_t n_slots, int32_t* starts,
                  int32_t* lens_out, int32_t* n_free_out, int32_t* status, int32_t* work, void* stream) {
    if (!lens || !more || !table || !n_free || !starts || !lens_out || !n_free_out || !status) return WB_EINVAL;
    if (n_slots < 0 || (n_slots > 0 && !slots) || free_size < 0 || (free_size > 0 && !free_pages)) return WB_EINVAL;
    const int v = check_table(R, width, page);
    if (v) return v;
    if (n_slots > 0x7FFFFFFF) return WB_EUNSUPPORTED;
    if (wb::plan_work(R, n_slots, lens_out == lens || n_free_out == n_free) && !work) return WB_EINVAL;
    if (!aligned(slots, 16)) return WB_EALIGN;
    for (const void* p : {(const void*)lens, (const void*)more, (const void*)table, (const void*)free_pages,
                          (const void*)n_free, (const void*)starts, (const void*)lens_out, (const void*)n_free_out,
                          (const void*)status, (const void*)work})
        if (!aligned(p, 4)) return WB_EALIGN;
    wb::PlanArgs a;
    a.lens = lens;
    a.more = more;
    a.table = table;
    a.free_pages = free_pages;
    a.n_free = n_free;
    a.slots = slots;
    a.starts = starts;
    a.lens_out = lens_out;
    a.n_free_out = n_free_out;
    a.status = status;
    a.work = work;
    a.R = R;
    a.width = width;
    a.free_size = free_size;
    a.page_log2 = page_log2(page);
    a.n_slots = n_slots;
    return hip_status(wb::launch_plan(a, static_cast<hipStream_t>(stream)));
}

int kv_release_pages(const uint8_t* ended, int32_t* lens, int R, const int32_t* table, int width, int32_t* free_pages,
                     int free_size, int32_t* n_free, int page, int32_t* status, void* stream) {
    if (!ended || !lens || !table || !n_free || !status) return WB_EINVAL;
    if (free_size < 0 || (free_size > 0 && !free_pages)) return WB_EINVAL;
    const int v = check_table(R, width, page);
    if (v) return v;
    for (const void* p : {(const void*)lens, (const void*)table, (const void*)free_pages, (const void*)n_free,
                          (const void*)status})
        if (!aligned(p, 4)) return WB_EALIGN;
    wb::ReleaseArgs a;
    a.ended = ended;
    a.lens = lens;
    a.table = table;
    a.free_pages = free_pages;
    a.n_free = n_free;
    a.status = status;
    a.R = R;
    a.width = width;
    a.free_size = free_size;
    a.page_log2 = page_log2(page);
    return hip_status(wb::launch_release(a, static_cast<hipStream_t>(stream)));
}

int kv_append(const wb_kv_cache* c, const void* k, const void* v, int64_t k_row, int64_t v_row, int src,
              const int64_t* slots, int N, void* stream) {
    const int s = check_cache(c);
    if (s) return s;
    if (N < 0) return WB_EINVAL;
    if (src != WB_F32 && src != c->dtype && !(c->dtype == WB_E4M3 && (src == WB_BF16 || src == WB_F16)))
        return src < WB_BF16 || src > WB_E4M3 ? WB_EINVAL : WB_EUNSUPPORTED;
    if (src == WB_E4M3) return WB_EUNSUPPORTED;
    if (N == 0) return WB_OK;
    if (!k || !v || !slots) return WB_EINVAL;
    if (int64_t(N) * c->H > 0x7FFFFFFF) return WB_EUNSUPPORTED;
    const int64_t row = int64_t(c->H) * c->D;
    if (N > 1 && (k_row < row || v_row < row)) return WB_EINVAL;
    const int size = element_size(src);
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || (N > 1 && ((k_row * size) % 16 || (v_row * size) % 16)))
        return WB_EALIGN;
    wb::AppendArgs a;
    a.c = *c;
    a.k = k;
    a.v = v;
    a.k_row = k_row;
    a.v_row = v_row;
    a.slots = slots;
    a.src = src;
    a.N = N;
    a.page_log2 = page_log2(c->page);
    return hip_status(wb::launch_append(a, static_cast<hipStream_t>(stream)));
}

int kv_attend_work(const wb_kv_cache* c, int R, int Hq, int width, size_t* bytes) {
    if (!bytes) return WB_EINVAL;
    const int v = check_attend(c, R, Hq, width);
    if (v) return v;
    // (either type of q: the one with more workgroups)
    *bytes = work_bytes_of(wb::attend_plan(*c, R, Hq, width, WB_BF16));
    return WB_OK;
}

int kv_attend(const wb_kv_cache* c, const void* q, int64_t q_row, int64_t q_head, int q_dtype, int R, int Hq,
              const int32_t* table, int width, const int32_t* lens, float scale, int window, void* o, float* lse,
              void* work, size_t work_bytes, void* stream) {
    const int v = check_attend(c, R, Hq, width);
    if (v) return v;
    if (!q || !table || !lens || !o || window < 0) return WB_EINVAL;
    if (q_dtype != WB_BF16 && q_dtype != WB_F16) return WB_EINVAL;
    if (c->dtype != WB_E4M3 && q_dtype != c->dtype) return WB_EUNSUPPORTED;
    if (!aligned(q, 16) || !aligned(o, 16) || q_row % 8 || q_head % 8 || !aligned(table, 4) || !aligned(lens, 4) ||
        !aligned(lse, 4))
        return WB_EALIGN;
    const wb::AttendPlan p = wb::attend_plan(*c, R, Hq, width, q_dtype);
    const size_t need = work_bytes_of(p);
    if (need) {
        if (!work) return WB_EINVAL;
        if (work_bytes < need) return WB_ESIZE;
        if (!aligned(work, 16)) return WB_EALIGN;
    }
    if (o == q) return WB_EINVAL;      // (a split request's query is read where another part has finished)
    wb::AttendArgs a;
    a.c = *c;
    a.q = q;
    a.q_row = q_row;
    a.q_head = q_head;
    a.table = table;
    a.lens = lens;
    a.o = o;
    a.lse = lse;
    if (need) {
        uint8_t* w = static_cast<uint8_t*>(work);
        a.part_o = reinterpret_cast<float*>(w);
        a.part_ml = reinterpret_cast<float*>(w + p.part_o_bytes);
        w += p.part_o_bytes + p.part_ml_bytes;
        if (p.joins_itself) {
            a.arrivals = reinterpret_cast<uint64_t*>(w + p.spans_bytes);
            a.tag = next_tag();
        } else {
            a.spans = reinterpret_cast<int64_t*>(w);
        }
    }
    a.scale = scale;
    a.R = R;
    a.Hq = Hq;
    a.width = width;
    a.window = window;
    a.q_dtype = q_dtype;
    a.page_log2 = page_log2(c->page);
    a.G = Hq / c->H;
    a.head_blocks = p.head_blocks;
    a.groups = p.groups;
    return hip_status(wb::launch_attend(a, static_cast<hipStream_t>(stream)));
}

int norm_quant(const void* x, int64_t x_row, const void* residual, int64_t r_row, void* residual_out, int64_t ro_row,
               const void* weight, int dtype, int N, int D, float eps, int group, uint8_t* codes, int64_t c_row,
               float* scales, void* stream) {
    if (dtype != WB_BF16 && dtype != WB_F16 && dtype != WB_F32) return WB_EINVAL;
    if (N < 0 || D < 1 || (residual != nullptr) != (residual_out != nullptr)) return WB_EINVAL;
    if (!(eps >= 0.f)) return WB_EINVAL;
    if (group != 0 && group != 128) return WB_EUNSUPPORTED;
    if (D > kMaxColumns) return WB_EUNSUPPORTED;
    if (N == 0) return WB_OK;
    if (!x || !codes || !scales) return WB_EINVAL;
    if (N > 1 && (x_row < D || c_row < D || (residual && (r_row < D || ro_row < D)))) return WB_EINVAL;
    if (residual && residual == residual_out && N > 1 && r_row != ro_row) return WB_EINVAL;
    const unsigned size = unsigned(element_size(dtype));
    if (!aligned(x, size) || !aligned(residual, size) || !aligned(residual_out, size) || !aligned(weight, size) ||
        !aligned(scales, 4))
        return WB_EALIGN;
    wb::NormArgs a;
    a.x = x;
    a.residual = residual;
    a.residual_out = residual_out;
    a.weight = weight;
    a.codes = codes;
    a.scales = scales;
    a.x_row = x_row;
    a.r_row = r_row;
    a.ro_row = ro_row;
    a.c_row = c_row;
    a.dtype = dtype;
    a.N = N;
    a.D = D;
    a.group = group;
    a.eps = eps;
    return hip_status(wb::launch_norm(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
