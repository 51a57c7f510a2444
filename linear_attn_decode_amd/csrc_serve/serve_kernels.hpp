// Kernel argument blocks and launch entry points of the serving operators (wbserve.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wbserve.h"

namespace wb {

// Work-items of one launch of the kernels that take some for each row or vector, at most: a grid's
// dimension holds fewer than 2^32. More rows go in several launches.
constexpr int64_t kLaunchItems = int64_t(1) << 31;

struct PlanArgs {
    const int32_t* lens = nullptr;
    const int32_t* more = nullptr;
    int32_t* table = nullptr;
    const int32_t* free_pages = nullptr;
    const int32_t* n_free = nullptr;
    int64_t* slots = nullptr;
    int32_t* starts = nullptr;
    int32_t* lens_out = nullptr;
    int32_t* n_free_out = nullptr;
    int32_t* status = nullptr;
    int32_t* work = nullptr;      // [R] pages taken before each request (plans of many slots)
    int R = 0, width = 0, free_size = 0, page_log2 = 0;
    int64_t n_slots = 0;
};
// int32 values of workspace; in_place: lens_out is lens, or n_free_out is n_free
int plan_work(int R, int64_t n_slots, bool in_place);
hipError_t launch_plan(const PlanArgs& a, hipStream_t stream);

struct ReleaseArgs {
    const uint8_t* ended = nullptr;
    int32_t* lens = nullptr;
    const int32_t* table = nullptr;
    int32_t* free_pages = nullptr;
    int32_t* n_free = nullptr;
    int32_t* status = nullptr;
    int R = 0, width = 0, free_size = 0, page_log2 = 0;
};
hipError_t launch_release(const ReleaseArgs& a, hipStream_t stream);

struct AppendArgs {
    wb_kv_cache c = {};
    const void* k = nullptr;
    const void* v = nullptr;
    int64_t k_row = 0, v_row = 0;
    const int64_t* slots = nullptr;
    int src = 0, N = 0, page_log2 = 0;
};
hipError_t launch_append(const AppendArgs& a, hipStream_t stream);

struct AttendArgs {
    wb_kv_cache c = {};
    const void* q = nullptr;
    int64_t q_row = 0, q_head = 0;
    const int32_t* table = nullptr;
    const int32_t* lens = nullptr;
    void* o = nullptr;
    float* lse = nullptr;
    float* part_o = nullptr;      // [groups][2][16][D] sums of unfinished segments
    float* part_ml = nullptr;     // [groups][2][16][2] their maximum and weight sum
    int64_t* spans = nullptr;     // [R + 1] first unit of each request, all units (for a second launch)
    uint64_t* arrivals = nullptr; // [groups] workgroups that stored a part of the segment that begins in
                                  // a workgroup's run and goes on behind it (or null: a second launch joins)
    uint64_t tag = 0;             // of this call, 52 bits, not 0
    float scale = 0.f;
    int R = 0, Hq = 0, width = 0, window = 0, q_dtype = 0, page_log2 = 0;
    int G = 1;                    // query heads of a key-value head
    int head_blocks = 1;          // key-value heads times blocks of 16 of their query heads
    int groups = 0;               // workgroups
};
struct AttendPlan {
    int head_blocks, groups;
    size_t part_o_bytes, part_ml_bytes, spans_bytes, arrivals_bytes;     // all 0: no request can take two turns
    bool joins_itself;                                   // the workgroups join what they split
};
AttendPlan attend_plan(const wb_kv_cache& c, int R, int Hq, int width, int q_dtype);
hipError_t launch_attend(const AttendArgs& a, hipStream_t stream);

struct ChunkArgs {
    wb_kv_cache c = {};
    const void* q = nullptr;
    int64_t q_row = 0, q_head = 0;
    const int32_t* table = nullptr;
    const int32_t* lens = nullptr;
    const int32_t* starts = nullptr;
    void* o = nullptr;
    float* lse = nullptr;
    float* part_o = nullptr;      // [slots][128][D] sums of the parts of split blocks
    float* part_ml = nullptr;     // [slots][128][2] their maximum and weight sum
    int64_t* before = nullptr;    // [R + 2] parts of the requests before each, tiles of a part (more than 64 requests)
    float scale = 0.f;
    int N = 0, R = 0, Hq = 0, width = 0, window = 0, q_dtype = 0, page_log2 = 0;
    int G = 1;                    // query heads of a key-value head
    int heads = 1, tokens = 1;    // of a block of rows: query heads of new tokens
    int head_blocks = 1;          // blocks of a key-value head's query heads
    int limbs = 2;                // 16-bit values that a weight enters the second product as
    int tile_log2 = 6;            // of the tokens of a key tile
    int part_tiles = 1;           // key tiles of a part at least
    int target = 1;               // parts that all tiles are cut into, about
    int64_t slots = 0, groups = 0, launched = 0;     // workgroups in all, and in the launches before
};
struct ChunkPlan {
    int heads, tokens, head_blocks, tile_log2, part_tiles, target;
    int64_t slots, groups;        // parts of split blocks at most (0: nothing is split); workgroups
    size_t part_o_bytes, part_ml_bytes, before_bytes;
};
ChunkPlan chunk_plan(const wb_kv_cache& c, int N, int R, int Hq, int width);
hipError_t launch_chunk(const ChunkArgs& a, hipStream_t stream);

struct RotateArgs {
    wb_heads q = {}, k = {};
    const void* positions = nullptr;
    const double* freqs = nullptr;
    float magnitude = 1.f, eps = 0.f;
    int dtype = 0, D = 0, rot = 0;
    bool wide = false;            // 64-bit positions
    bool interleaved = false;
    bool past = false;            // outputs past the caches
    int lanes = 4;                // of a head
    int waves_per_token = 1;
    int64_t first = 0, last = 0;  // tokens of the launch
};
hipError_t launch_rotate(RotateArgs a, int N, hipStream_t stream);

struct LogprobArgs {
    const void* logits = nullptr;
    int64_t row = 0;
    const void* tokens = nullptr;
    float* logprob = nullptr;
    float* entropy = nullptr;
    int32_t* top_ids = nullptr;
    float* top_logprobs = nullptr;
    uint64_t* parts = nullptr;    // [rows][segments][2 + K] sums and top keys of segments
    uint64_t* arrivals = nullptr; // [rows] segments stored
    uint64_t tag = 0;             // of this call, as for AttendArgs
    float scale = 1.f;
    int dtype = 0, V = 0, K = 0, segments = 1;
    int chunk = 1;                // vectors of a lane in a chunk
    int group = 8;                // vectors of a group whose maximum is kept
    bool wide = false;            // 64-bit tokens
    int64_t first = 0;            // row of the launch
};
struct LogprobPlan {
    int segments, chunk, group;
    size_t part_bytes, arrivals_bytes;
};
LogprobPlan logprob_plan(int N, int V, int K);
hipError_t launch_logprobs(LogprobArgs a, int N, hipStream_t stream);

struct NormArgs {
    const void* x = nullptr;
    const void* residual = nullptr;
    void* residual_out = nullptr;
    const void* weight = nullptr;
    uint8_t* codes = nullptr;
    float* scales = nullptr;
    int64_t x_row = 0, r_row = 0, ro_row = 0, c_row = 0;
    int dtype = 0, N = 0, D = 0, group = 0;
    float eps = 0.f;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);

}  // namespace wb
