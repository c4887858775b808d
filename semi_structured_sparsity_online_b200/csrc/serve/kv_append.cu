// New tokens' K and V into the 8-bit paged cache: one scale per (page, head).
//
//   s_tok = RN(amax over the page's new tokens / qmax)     qmax 127 (INT8), 448 (E4M3)
//   s     = max(s_old, s_tok)  where the page holds older tokens, else s_tok
//   code  = the library's code of RN(x / s); older codes, where s grew, the
//           code of RN(RN(code_old s_old) / s)
//
// The older tokens' values are known only as their codes, so a page whose
// scale grows rounds them once more; a page written in one call is rounded
// once. One CTA serves one (page, head) of K or of V: its new tokens are read
// once into registers, reduced to their amax and written as codes. Bound by
// memory: 2 (bf16) or 4 bytes read and 1 written per element.
#include "serve.cuh"

namespace ss24 {

namespace {

// 8 elements as they lie in memory
template <bool F32> struct Raw8 {
    uint4 w[F32 ? 2 : 1];
};
template <bool F32> __device__ __forceinline__ void load8(const void *base, int64_t at, Raw8<F32> &r)
{
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + at * (F32 ? 4 : 2));
    r.w[0] = __ldg(x);
    if constexpr (F32)
        r.w[1] = __ldg(x + 1);
}
template <bool F32> __device__ __forceinline__ void values8(const Raw8<F32> &r, float (&v)[8])
{
    if constexpr (F32) {
        const uint32_t u[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __uint_as_float(u[i]);
    } else {
        const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ float quotient(float v, const Recip &r)
{
    if (r.fast)
        return div_fast(v, r);
    return r.b > 0.0f ? __fdiv_rn(v, r.b) : 0.0f;
}

// Codes of 8 values. CLAMP: where a quotient may lie beyond the largest code (a
// scale outside the corrected reciprocal's range is a rounded subnormal; a code
// that no quantizer wrote). Else |x / s| <= qmax (1 + 2^-23), which rounds to qmax.
template <bool FP8, bool CLAMP> __device__ __forceinline__ uint2 encode8(const float (&v)[8], const Recip &r)
{
    uint32_t w[2] = {0, 0};
    if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i >> 1] |= static_cast<uint32_t>(cvt_e4m3x2h(quotient(v[2 * i], r), quotient(v[2 * i + 1], r))) << (16 * (i & 1));
    } else {
        // q + 1.5 2^23 holds the nearest integer (ties to even) in its low bits
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float q = quotient(v[i], r);
            if constexpr (CLAMP)
                q = fminf(fmaxf(q, -127.0f), 127.0f);
            c[i] = __float_as_uint(__fadd_rn(q, 12582912.0f));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
    }
    return make_uint2(w[0], w[1]);
}

template <bool FP8> __device__ __forceinline__ void decode8(uint2 c, float s, float (&v)[8])
{
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = (w[i >> 2] >> (8 * (i & 3))) & 0xff;
        const float x = FP8 ? e4m3_to_f32(b) : static_cast<float>(static_cast<int8_t>(b));
        v[i] = __fmul_rn(x, s);
    }
}

// CPT: chunks of 8 elements a thread holds, the most new ones of a page over the
// block's T threads.
template <bool FP8, bool F32, int CPT, int T>
__global__ void __launch_bounds__(T) kv_append_kernel(const KvAppendParams p)
{
    __shared__ float warp_max[T / 32];
    const KvCache &c = p.cache;
    const int h = blockIdx.y, kv = blockIdx.z;
    const uint32_t s = blockIdx.x / static_cast<uint32_t>(p.page_slots), slot = blockIdx.x - s * p.page_slots;
    grid_dependents_launch();
    grid_dependency_wait();

    int32_t first, count, len;
    if (!kv_sequence(p.batch, s, p.err, &first, &count, &len) || count == 0)
        return;
    const int32_t begin = len - count; // negative: the first tokens have no place
    const int32_t pi = ((begin > 0 ? begin : 0) >> c.log2_page) + static_cast<int32_t>(slot);
    const int64_t p0 = static_cast<int64_t>(pi) << c.log2_page;
    const int64_t lo = begin > p0 ? begin : p0, hi = len < p0 + c.page ? len : p0 + c.page;
    if (lo >= hi)
        return;
    const int32_t id = __ldg(p.batch.table + s * p.batch.table_ld + pi);
    const int fill = static_cast<int>(lo - p0), end = static_cast<int>(hi - p0); // new slots [fill, end)
    const HeadRows &x = p.x[kv];
    const int64_t row0 = first + (p0 - begin); // the token at slot 0
    const int lg_cpr = c.d == 128 ? 4 : 3;     // chunks per token

    const int chunks = (end - fill) << lg_cpr; // new ones

    // the tokens are on their way before the page number is looked at
    Raw8<F32> raw[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int ch = threadIdx.x + i * T;
        if (ch < chunks)
            load8<F32>(x.x, (row0 + fill + (ch >> lg_cpr)) * x.token_ld + h * x.head_ld + 8 * (ch & ((1 << lg_cpr) - 1)), raw[i]);
        else
            raw[i] = Raw8<F32>{};
    }
    if (id < 0 || id >= c.pages) {
        if (threadIdx.x == 0)
            atomicCAS(p.err, 0, kErrPage);
        return;
    }
    const int64_t page_head = static_cast<int64_t>(id) * c.kv_heads + h;
    uint8_t *codes = c.codes[kv] + (page_head << c.log2_page) * c.d;
    const float had = fill > 0 ? c.scales[kv][page_head] : 0.0f;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        float v[8];
        values8<F32>(raw[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            amax = fmaxf(amax, fabsf(v[j]));
    }
    for (int o = 16; o; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    if ((threadIdx.x & 31) == 0)
        warp_max[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 32; ++w)
        amax = fmaxf(amax, warp_max[w]);
    const float s_new = fmaxf(had, __fdiv_rn(amax, FP8 ? 448.0f : 127.0f));
    const Recip r = make_recip(s_new);
    if (threadIdx.x == 0)
        c.scales[kv][page_head] = s_new;
    uint2 *at = reinterpret_cast<uint2 *>(codes) + (fill << lg_cpr);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int ch = threadIdx.x + i * T;
        if (ch < chunks) {
            float v[8];
            values8<F32>(raw[i], v);
            at[ch] = r.fast ? encode8<FP8, false>(v, r) : encode8<FP8, true>(v, r);
        }
    }
    if (fill > 0 && s_new > had) {
        // the older codes, for the scale that grew
        at = reinterpret_cast<uint2 *>(codes);
#pragma unroll 4
        for (int ch = threadIdx.x; ch < fill << lg_cpr; ch += T) {
            float v[8];
            decode8<FP8>(at[ch], had, v);
            at[ch] = encode8<FP8, true>(v, r);
        }
    }
}

// Four chunks a thread where the page has them, in CTAs of 64 to 256 threads: small
// ones hide each other's start and barrier (8192 tokens, 8 heads of 128, bf16 to
// INT8: 12.5 us for pages of 16, 32 and 64, 3.9 TB/s; with 256 threads throughout
// 21.5, 16.6 and 13.0). Single tokens take 64 threads: 256 sequences 4.8 us, with
// 256 threads 15.5.
struct AppendShape {
    const void *kernel;
    int threads;
};
template <bool FP8, bool F32> AppendShape append_shape(int64_t chunks)
{
    if (chunks <= 64)
        return {reinterpret_cast<const void *>(kv_append_kernel<FP8, F32, 1, 64>), 64};
    if (chunks <= 256)
        return {reinterpret_cast<const void *>(kv_append_kernel<FP8, F32, 4, 64>), 64};
    if (chunks <= 512)
        return {reinterpret_cast<const void *>(kv_append_kernel<FP8, F32, 4, 128>), 128};
    if (chunks <= 1024)
        return {reinterpret_cast<const void *>(kv_append_kernel<FP8, F32, 4, 256>), 256};
    return {reinterpret_cast<const void *>(kv_append_kernel<FP8, F32, 8, 256>), 256};
}

} // namespace

cudaError_t launch_kv_append(const KvAppendParams &p, int x_f32, cudaStream_t stream)
{
    // the most new chunks of a page: at most 128 tokens of 16
    const int64_t chunks = (p.batch.max_new < p.cache.page ? p.batch.max_new : p.cache.page) * (p.cache.d / 8);
    const AppendShape shape =
        p.cache.fp8 ? (x_f32 ? append_shape<true, true>(chunks) : append_shape<true, false>(chunks))
                    : (x_f32 ? append_shape<false, true>(chunks) : append_shape<false, false>(chunks));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch.seqs * p.page_slots), static_cast<unsigned>(p.cache.kv_heads), 2);
    cfg.blockDim = dim3(shape.threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KvAppendParams pp = p;
    void *args[1] = {&pp};
    return cudaLaunchKernelExC(&cfg, shape.kernel, args);
}

} // namespace ss24
