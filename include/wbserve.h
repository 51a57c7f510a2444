/*
 * wbserve.h -- C ABI of the serving operators around the recurrent-state layers of a
 * hybrid language model (MI355X, gfx950): the paged key-value cache of its
 * full-attention layers (norms and rotary positions of queries and keys, page planning,
 * cache writes, attention of one new token and of chunks of them), the root-mean-square
 * norm whose output is stored in 8 bits, and log probabilities of tokens.
 *
 * Conventions are those of wbstate.h: status codes WB_*, caller-owned device memory (the
 * library never allocates), arguments validated on the host before anything is enqueued,
 * asynchronous execution on `stream` (a hipStream_t of the current device, which must be
 * the device of every pointer). No call synchronises the host, keeps anything of its inputs
 * or outputs for the next or uses device memory that was not passed to it, so calls on
 * different streams are independent and every call can be captured into a graph; what a
 * captured call reads (lengths, page tables, free pages) may change between replays. (The
 * process counts the calls of kv_attend and token_logprobs: a call marks its workspace with its number.)
 *
 * Stored keys and values: one array each, [pages][H][page][D], D contiguous: the tokens
 * of a page are contiguous for each key-value head. Token t of request r is token
 * t % page of page table[r][t / page]; its slot is table[r][t / page] * page + t % page.
 * 8-bit caches (WB_E4M3: 1-4-3 floating point without infinities, largest value 448) keep
 * a float32 scale for each stored vector, [pages][H][page]; a stored value stands for
 * code * scale.
 */
#ifndef WBSERVE_H
#define WBSERVE_H

#include "wbstate.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define WB_BF16 0
#define WB_F16 1
#define WB_F32 2
#define WB_E4M3 3
/* added to kv_attend_chunk's q_dtype: weights as one 16-bit value, not two */
#define WB_ONE_LIMB 256

/* A key-value cache in caller-owned device memory, 16-byte aligned. D is 64, 128 or 256;
 * page a power of two from 8 to 4096; dtype WB_BF16, WB_F16 or WB_E4M3 (then k_scale and
 * v_scale are set, else NULL); pages * page < 2^31. */
typedef struct wb_kv_cache {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t pages;
    int32_t page, H, D, dtype;
} wb_kv_cache;

/* Block tables and slot maps from request lengths. Request r holds lens[r] stored tokens
 * in the pages table[r][0 .. ceil(lens[r] / page)) and gets more[r] >= 0 new ones; the
 * pages they need beyond those held are popped off the stack of free pages free[0 ..
 * *n_free), topmost first, request by request:
 *   have_r = ceil(lens[r] / page), want_r = ceil((lens[r] + more[r]) / page),
 *   first_r = sum_{r' < r} (want_r' - have_r'),
 *   table[r][have_r + j] = free[*n_free - 1 - first_r - j], 0 <= j < want_r - have_r,
 *   starts[r] = sum_{r' < r} more[r'] (r = 0 .. R),
 *   slots[starts[r] + i] = slot of token lens[r] + i of request r; -1 in slots[starts[R] ..),
 *   lens_out[r] = lens[r] + more[r], *n_free_out = *n_free - sum_r (want_r - have_r),
 *   *status = 0.
 * lens_out may be lens and n_free_out may be n_free. Other table entries and the free
 * array are not written. lens, more, lens_out: int32 [R]; table: int32 [R][width];
 * free: int32 [free_size]; starts: int32 [R + 1]; slots: int64 [n_slots], 16-byte aligned;
 * n_free, n_free_out, status: int32 [1]; work: int32 [R], needed when kv_plan_work() says so.
 * All or nothing: a plan that cannot be carried out sets *status to the first of
 *   1  a negative length, a negative count of new tokens, or *n_free outside [0, free_size]
 *   2  a request would need more than `width` pages
 *   3  more new tokens than n_slots
 *   4  fewer free pages than needed
 * and then every slot is -1, starts is 0, lens_out = lens, *n_free_out = *n_free and the
 * table is left alone. (An entry of `free` is a page id that the library copies; the calls
 * that use page ids check them.) 1 <= R <= 65536; width * page at most 2^30, n_slots and
 * R * width below 2^31. */
int kv_plan_pages(const int32_t* lens, const int32_t* more, int R, int32_t* table, int width, const int32_t* free_pages,
                  int free_size, const int32_t* n_free, int page, int64_t* slots, int64_t n_slots, int32_t* starts,
                  int32_t* lens_out, int32_t* n_free_out, int32_t* status, int32_t* work, void* stream);

/* int32 values of workspace that kv_plan_pages needs (0: `work` may be NULL); in_place: whether
 * lens_out is lens or n_free_out is n_free. Host only. */
int kv_plan_work(int R, int64_t n_slots, int in_place);

/* Requests with ended[r] != 0 (uint8 [R]) give their ceil(lens[r] / page) pages back: they
 * are pushed onto the stack of free pages in the order of (request, page), *n_free grows by
 * their number and lens[r] becomes 0; table entries are left as they were. *status is 0, or,
 * with nothing changed, 1 for a negative length or *n_free outside [0, free_size], 2 for a
 * request of more than `width` pages, 4 if the pages would not fit into free_size. */
int kv_release_pages(const uint8_t* ended, int32_t* lens, int R, const int32_t* table, int width, int32_t* free_pages,
                     int free_size, int32_t* n_free, int page, int32_t* status, void* stream);

/* Writes the keys and values of N tokens, k and v [N][H][D] of type `src` with row strides
 * k_row and v_row (elements; heads and D contiguous), at slots[i] (int64) of the cache. A
 * slot outside [0, pages * page) is not stored (-1: padding). `src` is the cache's type or
 * WB_F32 (rounded to nearest), for an 8-bit cache also WB_BF16 or WB_F16: then
 * scale = max|x| / 448 (2^-126 at least) and code = e4m3(x / scale), to nearest with ties to
 * the even code; a vector of zeros has scale 0, one that holds a NaN or an infinity reads
 * back as NaN. A slot is given at most once in a call (kv_plan_pages gives none twice): one
 * that is given twice holds a mixture of its tokens. Rows 16-byte aligned; N * H below 2^31. */
int kv_append(const wb_kv_cache* c, const void* k, const void* v, int64_t k_row, int64_t v_row, int src,
              const int64_t* slots, int N, void* stream);

/* Attention of one new token per request over its stored tokens: with n = lens[r],
 * t in [max(0, n - window), n) (window 0: all) and head h reading key-value head
 * h / (Hq / H),
 *   s_t = scale * q[r][h] . k_t,  o[r][h] = sum_t e^{s_t} v_t / sum_t e^{s_t},
 *   lse[r][h] = log sum_t e^{s_t} (float32 [R][Hq], or NULL).
 * Scores, maxima and sums are float32, the weights e^{s_t - max} (times the value's scale, for
 * an 8-bit cache) enter the product with v as two 16-bit limbs, within 2^-17 of each weight (and
 * for a float16 cache 2^-40 of the largest), o is rounded once. A request without tokens, or
 * whose scores are all -infinity, has o = 0 and lse = -infinity. Stored values outside the range
 * are not used, whatever they hold; a NaN inside it gives NaN, an infinity what the formula
 * gives or NaN. A request with a length outside [0, width * page], or a page id outside
 * [0, pages) in the range it reads, has o = lse = NaN. Results do not depend on timing: equal
 * calls give equal bits.
 * q [R][Hq][D] of type q_dtype (the cache's, or WB_BF16 / WB_F16 for an 8-bit cache), strides
 * q_row and q_head in elements, multiples of 8; o [R][Hq][D] contiguous, of q's type; q and o
 * 16-byte aligned; table int32 [R][width]; lens int32 [R]. `work` has kv_attend_work() bytes
 * (NULL if 0), 16-byte aligned, whatever they hold, and belongs to the call until it has run.
 * No output overlaps an input. 1 <= R <= 65536, Hq a multiple of H and at most 4096, width * page at most 2^30. */
int kv_attend(const wb_kv_cache* c, const void* q, int64_t q_row, int64_t q_head, int q_dtype, int R, int Hq,
              const int32_t* table, int width, const int32_t* lens, float scale, int window, void* o, float* lse,
              void* work, size_t work_bytes, void* stream);

/* Bytes of workspace of kv_attend. Host only. */
int kv_attend_work(const wb_kv_cache* c, int R, int Hq, int width, size_t* bytes);

/* Attention of chunks of new tokens over the requests' stored tokens, the new ones among them
 * (kv_append has stored them): whole prompts, parts of prompts, drafted tokens and single tokens
 * in one call. Request r's m = starts[r + 1] - starts[r] new tokens are rows starts[r] ..
 * starts[r + 1] - 1 of q and o and the last m of its n = lens[r] stored ones (starts and lens as
 * kv_plan_pages gives them): row starts[r] + i has position p = n - m + i, and head h, which reads
 * key-value head h / (Hq / H), sees t in [max(0, p + 1 - window), p] (window 0: [0, p]):
 *   s_t = scale * q[row][h] . k_t,  o[row][h] = sum_t e^{s_t} v_t / sum_t e^{s_t},
 *   lse[row][h] = log sum_t e^{s_t} (float32 [N][Hq], or NULL).
 * Scores, maxima and sums are float32 (a row whose weighted sum of values, of weights to 2^4, passes its range
 * has infinities). The weights e^{s_t - ref} (ref within 4 / log2(e) of the
 * running maximum; times the value's scale, for an 8-bit cache) enter the product with v as two 16-bit
 * limbs of the cache's type (bfloat16 for an 8-bit one): within 2^-16 of each weight in bfloat16, 2^-21
 * and 2^-36 of the largest in float16. With WB_ONE_LIMB added to q_dtype they enter as one (2^-8; 2^-11
 * and 2^-36 of the largest), but for a float16 q over an 8-bit cache: o then has an error of weights
 * as large as that of its own rounding, and prompts take a quarter less time (drafted tokens 4 %). o is
 * rounded once. A row whose scores are all -infinity has o = 0 and lse = -infinity. Stored values
 * that a row does not see leave no trace in it, whatever they hold; a NaN that it sees gives NaN,
 * an infinity what the formula gives or NaN. A request with a length outside [m, width * page] has
 * o = lse = NaN, and so has a row that sees a token of a page id outside [0, pages) (other rows of
 * its request may); entries of pages that no row sees (before a window) may hold anything. A request
 * whose starts decrease or leave [0, N] has no rows; rows of no request are left as they were. (Where
 * starts decrease, later requests may have rows of earlier ones as well: those hold the result of one of
 * them, or are left.) Other than that equal calls give equal bits.
 * q [N][Hq][D] of type q_dtype (the cache's, or WB_BF16 / WB_F16 for an 8-bit cache), strides
 * q_row and q_head in elements, multiples of 8; o [N][Hq][D] contiguous, of q's type; q and o
 * 16-byte aligned; table int32 [R][width]; lens int32 [R]; starts int32 [R + 1]. `work` has
 * kv_attend_chunk_work() bytes (NULL if 0), 16-byte aligned, whatever they hold, and belongs to
 * the call until it has run. No output overlaps an input. N >= 0, N * Hq below 2^31; R, Hq and
 * width as for kv_attend. */
int kv_attend_chunk(const wb_kv_cache* c, const void* q, int64_t q_row, int64_t q_head, int q_dtype, int N, int R, int Hq,
                    const int32_t* table, int width, const int32_t* lens, const int32_t* starts, float scale, int window,
                    void* o, float* lse, void* work, size_t work_bytes, void* stream);

/* Bytes of workspace of kv_attend_chunk. Host only. */
int kv_attend_chunk_work(const wb_kv_cache* c, int N, int R, int Hq, int width, size_t* bytes);

/* Heads of N tokens, read at x and written at out (which may be x, with the same strides): head h of
 * token i begins at element i * row + h * head and is contiguous; out_row and out_head likewise.
 * weight: of the norm (D values of the same type), or NULL: no norm. */
typedef struct wb_heads {
    const void* x;
    void* out;
    const void* weight;
    int64_t row, head, out_row, out_head;
    int32_t H, reserved;
} wb_heads;

/* Norms and rotary positions of queries and keys: for each head of q and (if not NULL) k
 *   y = x / sqrt(mean(x^2) + eps) * weight  (weight NULL: y = x),
 * and pairs (a, b) of its first `rot` columns, (y_i, y_{i + rot / 2}) or, interleaved,
 * (y_{2 i}, y_{2 i + 1}), become
 *   (a cos t - b sin t, a sin t + b cos t) * magnitude,  t = position * freqs[i]  (radians),
 * the others stay y. freqs: float64 [rot / 2], any: positions scaled for long contexts are other
 * frequencies and a magnitude. Angles are taken in 64 bits (positions up to 2^31 to 2^-20 of a radian), the
 * rest is float32, outputs are rounded once. Rows of any finite size have their norm (where squares
 * leave float32's range, it is taken of the scaled row); a row of zeros stays zeros. positions: int32 [N],
 * or int64 with positions64; both may be NULL if rot is 0 (norms alone). Types WB_BF16, WB_F16, WB_F32;
 * 1 <= D <= 1024, rot even, 0 <= rot <= D. Outputs overlap nothing but their own input. */
int qk_rotate(const wb_heads* q, const wb_heads* k, int dtype, int N, int D, const void* positions, int positions64,
              const double* freqs, int rot, int interleaved, float magnitude, float eps, void* stream);

/* Log probabilities of given tokens: for each of N rows x of V logits (type `dtype`, `row` elements apart)
 *   lse = log sum_j e^{scale x_j},  logprob = scale x_token - lse,  p_j = e^{scale x_j - lse},
 *   entropy = -sum_j p_j log p_j  (NULL: not wanted),
 *   top_ids, top_logprobs [N][K]: the K largest logits' columns and their log probabilities, larger logits
 *   first, equal ones by their column; NaN counts as -infinity in this order (K 0: not wanted).
 * Sums are float32, of differences from the largest logit, so that scale x may be of any size (log probabilities
 * past float32's range are -infinity); no log probability is above 0, no entropy below. A token outside [0, V)
 * (padding) has logprob NaN; logits of -infinity have p = 0; a row that holds a NaN or +infinity, or nothing
 * but -infinity, has NaN in place of its log probabilities and entropy. tokens: int32 [N], or int64 with tokens64. logprob, entropy: float32 [N]; top_ids int32,
 * top_logprobs float32. 1 <= V <= 2^24 (2^24 - 8 with K > 32), K <= 64 and V, 2^-100 <= scale <= 2^100 (1 / temperature), N >= 0.
 * `work` as for kv_attend, of token_logprobs_work() bytes. Equal calls give equal bits. No output overlaps an input. */
int token_logprobs(const void* logits, int64_t row, int dtype, int N, int V, const void* tokens, int tokens64, float scale,
                   float* logprob, float* entropy, int K, int32_t* top_ids, float* top_logprobs, void* work,
                   size_t work_bytes, void* stream);

/* Bytes of workspace of token_logprobs. Host only. */
int token_logprobs_work(int N, int V, int K, size_t* bytes);

/* Root-mean-square norm with an 8-bit output: for each of N rows of D columns
 *   h = x + residual (float32; residual NULL: h = x), residual_out = h rounded to residual's type,
 *   y = h / sqrt(mean(h^2) + eps) * weight (weight NULL: 1),
 *   scale_g = max_{j in group g} |y_j| / 448 (2^-126 at least), code_j = e4m3(y_j / scale_g),
 * groups of `group` columns (128; the last may be shorter) or the whole row (group 0). The
 * norm takes h before it is rounded, of any finite size (where its squares leave float32's
 * range, it takes h and eps scaled). x, residual, residual_out, weight are of type `dtype`
 * (WB_BF16, WB_F16, WB_F32); x_row, r_row, ro_row, c_row are row strides in elements; scales
 * float32 [N][ceil(D / group)]. A group of zeros has scale 0 and codes 0; a group that holds
 * a NaN or an infinity, or whose row holds a NaN, has NaN codes. residual_out may be
 * residual (same stride); nothing else may overlap. 1 <= D <= 65536, N >= 0. */
int norm_quant(const void* x, int64_t x_row, const void* residual, int64_t r_row, void* residual_out, int64_t ro_row,
               const void* weight, int dtype, int N, int D, float eps, int group, uint8_t* codes, int64_t c_row,
               float* scales, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WBSERVE_H */
