// Internal interface of the 8-bit serving operators: the INT8 product, the
// 8-bit paged cache and attention over it (abi_serve.cu checks the arguments;
// one file per operator).
#pragma once

#include "../device.cuh"
#include "../internal.cuh"

namespace ss24 {

// Error words of these kernels (workspace header; ss24.h documents them).
constexpr int32_t kErrGemmWait = 14;    // INT8 product: a barrier wait ran out
constexpr int32_t kErrAttendWait = 15;  // attention: a barrier wait ran out
constexpr int32_t kErrPage = 16;        // a page number outside the cache
constexpr int32_t kErrBatch = 17;       // starts / lengths against tokens, max_new or max_len

struct GemmInt8Params {
    int64_t m, n, k, ldy;
    const int8_t *a, *b;
    const float *a_scale, *b_scale;
    void *y;
    int32_t y_f32;
    int32_t *err;
    uint64_t wait_limit_ns;
    int32_t test_skip; // >= 0: a stage that the first CTA does not copy (ss24.h, test hook)
};

// The paged cache: codes [pages][kv_heads][page][d], scales [pages][kv_heads].
struct KvCache {
    uint8_t *codes[2];  // k, v
    float *scales[2];
    int64_t pages;
    int32_t kv_heads, page, log2_page, d, fp8;
};

// The sequences of a call: page numbers [seqs][table_ld], starts [seqs + 1]
// (new tokens of sequence s are rows starts[s] .. starts[s + 1] - 1), lengths
// [seqs] (tokens in the cache, the new ones included).
struct KvBatch {
    const int32_t *table, *starts, *lengths;
    int64_t seqs, table_ld, tokens, max_new, max_len;
};

// Per-token, per-head rows of d elements.
struct HeadRows {
    void *x;
    int64_t token_ld, head_ld;
};

struct KvAppendParams {
    KvCache cache;
    KvBatch batch;
    HeadRows x[2];      // k, v
    int64_t page_slots; // most pages a sequence's new tokens touch
    int32_t *err;
};

struct KvAttendParams {
    KvCache cache;
    KvBatch batch;
    HeadRows q, out;
    float *lse;          // [tokens][q_heads] or nullptr
    float scale_log2;    // softmax scale times log2(e)
    int32_t causal, group;
    int32_t row_tiles;   // row tiles of one (sequence, KV head)
    int32_t splits;      // parts of the key axis
    int32_t split_keys;  // keys in a part, a multiple of the key step
    float *part_o;       // [tokens * q_heads][splits][d] (splits > 1)
    float *part_lse;     // [tokens * q_heads][splits], base 2
    int32_t *err;
    uint64_t wait_limit_ns;
    int32_t test_skip; // >= 0: a round or step whose keys or values the first CTA does not hand over
};

cudaError_t launch_gemm_int8(const GemmInt8Params &p, cudaStream_t stream);
cudaError_t launch_kv_append(const KvAppendParams &p, int x_f32, cudaStream_t stream);
// Chooses the kernel and the parts of the key axis; fills p's row_tiles,
// splits and split_keys.
void kv_attend_plan(KvAttendParams *p);
cudaError_t launch_kv_attend(const KvAttendParams &p, cudaStream_t stream);

// A map of the [rows][row_bytes] byte matrix at base for boxes of box_bytes (64
// or 128, the swizzle's span too) x box_rows.
bool tensor_map_bytes(CUtensorMap *map, const void *base, int64_t rows, int64_t row_bytes, uint32_t box_bytes,
                      uint32_t box_rows);

// New tokens of sequence s and its length, checked against the call's bounds;
// false (and the error word) where they do not hold, which leaves the
// sequence out.
__device__ __forceinline__ bool kv_sequence(const KvBatch &b, int64_t s, int32_t *err, int32_t *first, int32_t *count,
                                            int32_t *len)
{
    const int32_t s0 = b.starts[s], s1 = b.starts[s + 1], l = b.lengths[s];
    *first = s0;
    *count = s1 - s0;
    *len = l;
    const bool ok = s0 >= 0 && s1 >= s0 && s1 <= b.tokens && s1 - s0 <= b.max_new && l >= 0 && l <= b.max_len;
    if (!ok)
        atomicCAS(err, 0, kErrBatch);
    return ok;
}

} // namespace ss24
