// The C ABI of the 8-bit serving operators (include/ss24.h): host-side checks
// and launches. Every check runs before anything is enqueued.
#include <cmath>
#include <cstdlib>

#include "../../../include/ss24.h"
#include "serve.cuh"

using namespace ss24;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

ss24_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SS24_OK : SS24_ERR_CUDA; }

ss24_status check_ws(const void *ws, size_t ws_bytes)
{
    return !ws || ws_bytes < kWsBytes || !aligned(ws, 256) ? SS24_ERR_WORKSPACE : SS24_OK;
}

int32_t *error_word(void *ws) { return reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + kWsErrOff); }

// The limit of the kernels' waits, and the test hook (ss24.h).
void wait_limits(uint64_t *limit_ns, int32_t *skip)
{
    *limit_ns = kWaitLimitNs;
    *skip = -1;
    if (const char *t = std::getenv("SS24_TEST_SKIP_TILE")) {
        const long v = std::strtol(t, nullptr, 10);
        if (v >= 0 && v < INT32_MAX) {
            *skip = static_cast<int32_t>(v);
            *limit_ns = kTestWaitLimitNs;
        }
    }
}

ss24_status check_cache(const ss24_kv_cache *c, KvCache *out)
{
    if (!c)
        return SS24_ERR_NULL;
    if (c->kind != SS24_FMT_INT && c->kind != SS24_FMT_FP8_E4M3)
        return SS24_ERR_FORMAT;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
        return SS24_ERR_SHAPE;
    if ((c->head_dim != 64 && c->head_dim != 128) || c->kv_heads < 1 || c->kv_heads > 1024 || c->pages < 0 ||
        c->pages > INT32_MAX / (static_cast<int64_t>(c->kv_heads) * c->page))
        return SS24_ERR_SHAPE;
    if (c->pages > 0 && (!c->k || !c->v || !c->k_scales || !c->v_scales))
        return SS24_ERR_NULL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))
        return SS24_ERR_ALIGN;
    int lg = 4;
    while ((1 << lg) < c->page)
        ++lg;
    *out = KvCache{{static_cast<uint8_t *>(c->k), static_cast<uint8_t *>(c->v)},
                   {c->k_scales, c->v_scales},
                   c->pages,
                   c->kv_heads,
                   c->page,
                   lg,
                   c->head_dim,
                   c->kind == SS24_FMT_FP8_E4M3};
    return SS24_OK;
}

ss24_status check_batch(const ss24_kv_batch *b, const KvCache &c, KvBatch *out)
{
    if (!b)
        return SS24_ERR_NULL;
    // lengths stay far enough below 2^31 that a key step past the end is an int32
    constexpr int64_t kMost = INT32_MAX - 65536;
    if (b->seqs < 0 || b->seqs > kMost || b->tokens < 0 || b->tokens > kMost || b->max_new < 0 ||
        b->max_new > b->tokens || b->max_len < 0 || b->max_len > kMost || b->table_ld < 0 || b->table_ld > kMost ||
        b->table_ld * c.page < b->max_len)
        return SS24_ERR_SHAPE;
    if (b->seqs > 0 && (!b->starts || !b->lengths || (b->max_len > 0 && !b->page_table)))
        return SS24_ERR_NULL;
    if (!aligned(b->starts, 4) || !aligned(b->lengths, 4) || !aligned(b->page_table, 4))
        return SS24_ERR_ALIGN;
    *out = KvBatch{b->page_table, b->starts, b->lengths, b->seqs, b->table_ld, b->tokens, b->max_new, b->max_len};
    return SS24_OK;
}

// Rows of head_dim elements, each 16-byte aligned.
ss24_status check_rows(const ss24_head_rows *r, int64_t head_dim, bool allow_f32, bool needed, HeadRows *out)
{
    if (!r || (!r->x && needed))
        return SS24_ERR_NULL;
    if (r->dtype != SS24_BF16 && !(allow_f32 && r->dtype == SS24_F32))
        return SS24_ERR_DTYPE;
    if (r->heads < 1 || r->token_stride < head_dim || (r->heads > 1 && r->head_stride < head_dim))
        return SS24_ERR_SHAPE;
    const int64_t es = r->dtype == SS24_BF16 ? 2 : 4;
    if (!aligned(r->x, 16) || (r->token_stride * es) % 16 != 0 || (r->heads > 1 && (r->head_stride * es) % 16 != 0))
        return SS24_ERR_ALIGN;
    *out = HeadRows{r->x, r->token_stride, r->heads > 1 ? r->head_stride : 0};
    return SS24_OK;
}

// The plan of an attention call; false where its grid would not fit.
bool plan_attention(const KvCache &c, const KvBatch &b, int32_t q_heads, KvAttendParams *p)
{
    p->cache = c;
    p->batch = b;
    p->group = q_heads / c.kv_heads;
    kv_attend_plan(p);
    const double ctas = static_cast<double>(b.seqs) * c.kv_heads * p->row_tiles * p->splits;
    return 2.0 * ctas < 2147483647.0 && static_cast<double>(b.tokens) * q_heads < 2147483647.0;
}

int64_t scratch_floats(const KvAttendParams &p)
{
    if (p.splits <= 1)
        return 0;
    const int64_t rows = p.batch.tokens * p.cache.kv_heads * p.group;
    return rows * p.splits * (p.cache.d + 1);
}

} // namespace

extern "C" {

ss24_status ss24_gemm_int8(const int8_t *a, const float *a_scale, const int8_t *b, const float *b_scale, int64_t m,
                           int64_t n, int64_t k, void *y, int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes,
                           ss24_stream stream)
{
    if (y_dtype != SS24_BF16 && y_dtype != SS24_F32)
        return SS24_ERR_DTYPE;
    // 128 * 128 * k < 2^31: the integer sum is exact for every code
    if (m < 0 || n < 0 || k <= 0 || m > INT32_MAX || n > INT32_MAX || k % 16 != 0 || k > 131071 || ldy < n)
        return SS24_ERR_SHAPE;
    ss24_status st = check_ws(ws, ws_bytes);
    if (st != SS24_OK)
        return st;
    if (m == 0 || n == 0)
        return SS24_OK;
    if (!a || !a_scale || !b || !b_scale || !y)
        return SS24_ERR_NULL;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4) ||
        !aligned(y, y_dtype == SS24_BF16 ? 2 : 4))
        return SS24_ERR_ALIGN;
    GemmInt8Params p{m, n, k, ldy, a, b, a_scale, b_scale, y, y_dtype == SS24_F32, error_word(ws)};
    wait_limits(&p.wait_limit_ns, &p.test_skip);
    return cuda_status(launch_gemm_int8(p, reinterpret_cast<cudaStream_t>(stream)));
}

ss24_status ss24_kv_append(const ss24_kv_cache *cache, const ss24_kv_batch *batch, const ss24_head_rows *k,
                           const ss24_head_rows *v, void *ws, size_t ws_bytes, ss24_stream stream)
{
    KvAppendParams p{};
    ss24_status st = check_cache(cache, &p.cache);
    if (st == SS24_OK)
        st = check_batch(batch, p.cache, &p.batch);
    if (st != SS24_OK)
        return st;
    const bool any = p.batch.seqs > 0 && p.batch.tokens > 0 && p.batch.max_new > 0 && p.batch.max_len > 0;
    const ss24_head_rows *x[2] = {k, v};
    for (int i = 0; i < 2; ++i) {
        st = check_rows(x[i], p.cache.d, true, any, &p.x[i]);
        if (st != SS24_OK)
            return st;
        if (x[i]->heads != p.cache.kv_heads)
            return SS24_ERR_SHAPE;
    }
    if (k->dtype != v->dtype)
        return SS24_ERR_DTYPE;
    st = check_ws(ws, ws_bytes);
    if (st != SS24_OK || !any)
        return st;
    // the new tokens may start on a page's last slot
    p.page_slots = (p.batch.max_new + p.cache.page - 2) / p.cache.page + 1;
    if (static_cast<double>(p.batch.seqs) * p.page_slots >= 2147483647.0)
        return SS24_ERR_SHAPE;
    p.err = error_word(ws);
    return cuda_status(launch_kv_append(p, k->dtype == SS24_F32, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t ss24_kv_attention_scratch_bytes(const ss24_kv_cache *cache, const ss24_kv_batch *batch, int32_t q_heads)
{
    KvAttendParams p{};
    if (check_cache(cache, &p.cache) != SS24_OK || check_batch(batch, p.cache, &p.batch) != SS24_OK || q_heads < 1 ||
        q_heads % p.cache.kv_heads != 0)
        return -1;
    if (p.batch.seqs == 0 || p.batch.tokens == 0 || p.batch.max_new == 0)
        return 0;
    if (!plan_attention(p.cache, p.batch, q_heads, &p))
        return -1;
    return 4 * scratch_floats(p);
}

ss24_status ss24_kv_attention(const ss24_head_rows *q, const ss24_kv_cache *cache, const ss24_kv_batch *batch,
                              float scale, int32_t causal, const ss24_head_rows *out, float *lse, void *scratch,
                              int64_t scratch_bytes, void *ws, size_t ws_bytes, ss24_stream stream)
{
    KvAttendParams p{};
    ss24_status st = check_cache(cache, &p.cache);
    if (st == SS24_OK)
        st = check_batch(batch, p.cache, &p.batch);
    if (st != SS24_OK)
        return st;
    const bool any = p.batch.seqs > 0 && p.batch.tokens > 0 && p.batch.max_new > 0;
    st = check_rows(q, p.cache.d, false, any, &p.q);
    if (st == SS24_OK)
        st = check_rows(out, p.cache.d, false, any, &p.out);
    if (st != SS24_OK)
        return st;
    if (q->heads != out->heads || q->heads % p.cache.kv_heads != 0)
        return SS24_ERR_SHAPE;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    if (!std::isfinite(p.scale_log2) || (causal != 0 && causal != 1))
        return SS24_ERR_ARG;
    if (!aligned(lse, 4))
        return SS24_ERR_ALIGN;
    st = check_ws(ws, ws_bytes);
    if (st != SS24_OK || !any)
        return st;
    if (!plan_attention(p.cache, p.batch, q->heads, &p))
        return SS24_ERR_SHAPE;
    const int64_t need = scratch_floats(p);
    if (need > 0 && (!scratch || scratch_bytes < 4 * need || !aligned(scratch, 16)))
        return SS24_ERR_WORKSPACE;
    p.lse = lse;
    p.causal = causal;
    p.part_o = static_cast<float *>(scratch);
    p.part_lse = p.part_o + need / (p.cache.d + 1) * p.cache.d;
    p.err = error_word(ws);
    wait_limits(&p.wait_limit_ns, &p.test_skip);
    return cuda_status(launch_kv_attend(p, reinterpret_cast<cudaStream_t>(stream)));
}

} // extern "C"
