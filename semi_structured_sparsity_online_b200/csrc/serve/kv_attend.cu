// Attention of new tokens over the 8-bit paged cache, few query rows per
// (sequence, KV head): one warp works on 16 keys at a time.
//
//   x[r][j] = scale q_r . (k_j s_k) log2(e),  s_k, s_v: the scales of j's page
//   o_r = sum_j 2^(x[r][j]) (v_j s_v) / sum_j 2^(x[r][j]),  lse_r = ln 2 log2 sum_j 2^(x[r][j])
//
// Rows. The queries of the heads that share a KV head (group) and of several
// new tokens are rows of one tile: row r is token r / group, head r % group.
// Both products run on the tensor cores with the keys (or the head dimension)
// as the MMA's M and 8 rows as its N, so that 4 or 8 rows leave nothing idle.
// The codes go from global memory to registers in 16-byte loads; the MMA's k
// order is free as long as both operands agree, so no shuffle or shared
// memory lies between a load and its MMA. Codes are exact in fp16 (|code| <=
// 127, or E4M3). q is held in fp16 after a power-of-two scaling of its row by
// its largest magnitude: what that drops is below 2^-24 of that magnitude.
//
// The weights of the second product carry the V scale: w = 2^(x + log2 s_v -
// M) with M a running bound on x + log2 s_v, so that w <= 2^8 fits fp16
// (rounded once, 2^-11 relative) and its small values are small next to the
// sum they enter. M moves only when a value exceeds it by 2^8. The denominator
// sums w / s_v in binary32. Scales s_v below 2^-100 count as 2^-100.
#include "kv_attend.cuh"

namespace ss24 {

namespace {

// bytes i of a and of b (i = 0..3) -> four fp16 pairs (a_i, b_i)
template <bool FP8> __device__ __forceinline__ void pairs4_to_f16(uint32_t a, uint32_t b, uint32_t (&out)[4])
{
    codes4_to_f16<FP8>(__byte_perm(a, b, 0x5140), out[0], out[1]);
    codes4_to_f16<FP8>(__byte_perm(a, b, 0x7362), out[2], out[3]);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint4 load_codes16(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A warp's 16 keys. Lane (g, q) = (lane / 4, lane % 4) holds, of K, keys g and
// g + 8: for D = 128 the 16 bytes at 64 c + 16 q, c = 0, 1 (D = 64: at 16 q);
// of V, the D / 8 bytes at g D / 8 of keys 2q, 2q + 1, 2q + 8, 2q + 9.
template <int D> struct Keys16 {
    uint4 k[2][D / 64];
    uint32_t v[4][D / 32];
    float ks, vs;
    bool there;
};

template <int D>
__device__ __forceinline__ void load_keys(Keys16<D> &t, const KvAttendParams &p, int32_t id, int h, int32_t key0,
                                          int lane)
{
    t.there = id >= 0 && id < p.cache.pages;
    if (!t.there)
        return;
    const int g = lane >> 2, q = lane & 3;
    const int64_t ph = static_cast<int64_t>(id) * p.cache.kv_heads + h;
    const int64_t at = ((ph << p.cache.log2_page) + (key0 & (p.cache.page - 1))) * D;
    const uint8_t *k = p.cache.codes[0] + at + g * D + 16 * q, *v = p.cache.codes[1] + at + 2 * q * D + g * (D / 8);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        t.k[0][c] = load_codes16(k + 64 * c);
        t.k[1][c] = load_codes16(k + 8 * D + 64 * c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t *at_i = v + ((i & 1) + 8 * (i >> 1)) * D;
        if constexpr (D == 128) {
            const uint4 w = load_codes16(at_i);
            t.v[i][0] = w.x, t.v[i][1] = w.y, t.v[i][2] = w.z, t.v[i][3] = w.w;
        } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(at_i));
            t.v[i][0] = w.x, t.v[i][1] = w.y;
        }
    }
    t.ks = __ldg(p.cache.scales[0] + ph);
    t.vs = __ldg(p.cache.scales[1] + ph);
}

// NT: n tiles of 8 rows; WARPS warps take turns on the part's 16-key steps.
template <int D, bool FP8, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) kv_attend_rows_kernel(const KvAttendParams p)
{
    constexpr int ROWS = 8 * NT, MT = D / 16;
    __shared__ float sm_o[WARPS][ROWS][D + 4];
    __shared__ float sm_m[WARPS][ROWS], sm_l[WARPS][ROWS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    int64_t b = blockIdx.x;
    const int split = static_cast<int>(b % p.splits);
    b /= p.splits;
    const int tile = static_cast<int>(b % p.row_tiles);
    b /= p.row_tiles;
    const int h = static_cast<int>(b % p.cache.kv_heads);
    const int64_t s = b / p.cache.kv_heads;
    grid_dependency_wait();

    int32_t first, count, len;
    const bool fine = kv_sequence(p.batch, s, p.err, &first, &count, &len);
    const int64_t row0 = static_cast<int64_t>(tile) * ROWS, rows = static_cast<int64_t>(count) * p.group;
    if (!fine || row0 >= rows)
        return;
    const int live = static_cast<int>(rows - row0 < ROWS ? rows - row0 : ROWS);
    // the part's keys, no further than the tile's last row sees
    int64_t kb = static_cast<int64_t>(split) * p.split_keys;
    int64_t ke = kb + p.split_keys;
    const int32_t last = row_at(p, row0 + live - 1, h, first, count, len).limit;
    if (ke > last)
        ke = last;

    // q: n tile t, row g: the 4 values of d that step ks of K's lane layout names
    uint32_t qf[NT][MT][2];
    float fac[NT][2];
    int32_t limit[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float v[MT][4];
        float amax = 0.0f;
        const int r = 8 * t + g;
        const bool on = r < live;
        const RowAt a = row_at(p, row0 + (on ? r : 0), h, first, count, len);
        const __nv_bfloat16 *src =
            static_cast<const __nv_bfloat16 *>(p.q.x) + a.token * p.q.token_ld + a.head * p.q.head_ld;
#pragma unroll
        for (int ks = 0; ks < MT; ++ks) {
            const uint2 w =
                __ldg(reinterpret_cast<const uint2 *>(src + (ks / 4) * 64 + 16 * q + 4 * (ks & 3)));
            v[ks][0] = on ? __uint_as_float(w.x << 16) : 0.0f;
            v[ks][1] = on ? __uint_as_float(w.x & 0xffff0000u) : 0.0f;
            v[ks][2] = on ? __uint_as_float(w.y << 16) : 0.0f;
            v[ks][3] = on ? __uint_as_float(w.y & 0xffff0000u) : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                amax = fmaxf(amax, fabsf(v[ks][i]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        // 2^-e with e the exponent of amax, kept to normal numbers
        int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
        e = e < -100 ? -100 : e > 100 ? 100 : e;
        const float down = exp2_int(-e);
#pragma unroll
        for (int ks = 0; ks < MT; ++ks) {
            qf[t][ks][0] = pack_f16(v[ks][0] * down, v[ks][1] * down);
            qf[t][ks][1] = pack_f16(v[ks][2] * down, v[ks][3] * down);
        }
        const float f = p.scale_log2 * exp2_int(e);
        // the accumulators' rows of this lane: 2q, 2q + 1
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            fac[t][i] = __shfl_sync(kFull, f, (2 * q + i) * 4);
            const int rr = 8 * t + 2 * q + i;
            limit[t][i] = rr < live ? row_at(p, row0 + rr, h, first, count, len).limit : 0;
        }
    }
    const int32_t low = row_at(p, row0, h, first, count, len).limit; // the least any row sees

    float o[NT][MT][4] = {};
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        m[t][0] = m[t][1] = -1e30f, l[t][0] = l[t][1] = 0.0f;

    const int32_t *table = p.batch.table + s * p.batch.table_ld;
    auto page_of = [&](int64_t key) { return key < ke ? __ldg(table + (key >> p.cache.log2_page)) : -1; };
    int64_t key = kb + 16 * warp;
    Keys16<D> next;
    load_keys<D>(next, p, page_of(key), h, static_cast<int32_t>(key), lane);
    int32_t id = page_of(key + 16 * WARPS);
    for (; key < ke; key += 16 * WARPS) {
        Keys16<D> cur = next;
        load_keys<D>(next, p, id, h, static_cast<int32_t>(key + 16 * WARPS), lane);
        id = page_of(key + 32 * WARPS);
        if (!cur.there) {
            if (lane == 0)
                atomicCAS(p.err, 0, kErrPage);
            continue;
        }
        float sc[NT][4] = {};
#pragma unroll
        for (int ks = 0; ks < MT; ++ks) {
            const uint4 wa = cur.k[0][ks / 4], wb = cur.k[1][ks / 4];
            const uint32_t a = (ks & 3) == 0 ? wa.x : (ks & 3) == 1 ? wa.y : (ks & 3) == 2 ? wa.z : wa.w;
            const uint32_t c = (ks & 3) == 0 ? wb.x : (ks & 3) == 1 ? wb.y : (ks & 3) == 2 ? wb.z : wb.w;
            uint32_t a0, a1, a2, a3;
            codes4_to_f16<FP8>(a, a0, a2);
            codes4_to_f16<FP8>(c, a1, a3);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                mma_f16(sc[t], a0, a1, a2, a3, qf[t][ks][0], qf[t][ks][1]);
        }
        // sc[t]: (key g, rows 2q, 2q + 1), (key g + 8, the same rows)
        const float sv = fmaxf(cur.vs, 0x1p-100f);
        const float lsv = log2f(sv), inv = __frcp_rn(sv);
        const bool edge = key + 16 > ke || key + 16 > low;
        bool above = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sc[t][i] = fmaf(sc[t][i], cur.ks * fac[t][i & 1], lsv);
                if (edge) {
                    const int32_t j = static_cast<int32_t>(key) + g + 8 * (i >> 1);
                    if (j >= limit[t][i & 1] || j >= ke)
                        sc[t][i] = -INFINITY;
                }
                above |= sc[t][i] > m[t][i & 1] + 8.0f;
            }
        if (__any_sync(kFull, above)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = fmaxf(sc[t][i], sc[t][i + 2]);
                    x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
                    x = fmaxf(x, m[t][i]);
                    const float f = exp2_approx(m[t][i] - x);
                    m[t][i] = x;
                    l[t][i] *= f;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        o[t][mt][i] *= f;
                        o[t][mt][i + 2] *= f;
                    }
                }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = exp2_approx(sc[t][i] - m[t][i & 1]);
            l[t][0] = fmaf(w[0] + w[2], inv, l[t][0]);
            l[t][1] = fmaf(w[1] + w[3], inv, l[t][1]);
            pf[t][0] = transpose8x8(pack_f16(w[0], w[1]));
            pf[t][1] = transpose8x8(pack_f16(w[2], w[3]));
        }
        if (FP8 && key + 16 > ke) {
            // slots behind the last token may hold NaN codes
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (key + 2 * q + (i & 1) + 8 * (i >> 1) >= ke)
#pragma unroll
                    for (int w = 0; w < D / 32; ++w)
                        cur.v[i][w] = 0;
        }
        // m tile mt: rows g, g + 8 are elements g D / 8 + 2 mt, + 1
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            uint32_t lo[4], hi[4];
            pairs4_to_f16<FP8>(cur.v[0][w], cur.v[1][w], lo);
            pairs4_to_f16<FP8>(cur.v[2][w], cur.v[3][w], hi);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                mma_f16(o[t][2 * w], lo[0], lo[1], hi[0], hi[1], pf[t][0], pf[t][1]);
                mma_f16(o[t][2 * w + 1], lo[2], lo[3], hi[2], hi[3], pf[t][0], pf[t][1]);
            }
        }
    }

    // the warps' sums joined
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[t][i] += __shfl_xor_sync(kFull, l[t][i], 4);
            l[t][i] += __shfl_xor_sync(kFull, l[t][i], 8);
            l[t][i] += __shfl_xor_sync(kFull, l[t][i], 16);
            const int r = 8 * t + 2 * q + i;
            if (g == 0)
                sm_m[warp][r] = m[t][i], sm_l[warp][r] = l[t][i];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                *reinterpret_cast<float2 *>(&sm_o[warp][r][g * (D / 8) + 2 * mt]) =
                    make_float2(o[t][mt][i], o[t][mt][i + 2]);
        }
    __syncthreads();
    for (int e = threadIdx.x; e < live * (D / 4); e += WARPS * 32) {
        const int r = e / (D / 4), d = 4 * (e % (D / 4));
        float top = -1e30f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            top = fmaxf(top, sm_m[w][r]);
        float den = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = exp2_approx(sm_m[w][r] - top);
            den = fmaf(f, sm_l[w][r], den);
            const float4 x = *reinterpret_cast<const float4 *>(&sm_o[w][r][d]);
            acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y);
            acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
        }
        const bool any = den > 0.0f;
        const float inv = any ? __frcp_rn(den) : 0.0f;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        const float lse2 = any ? top + log2f(den) : -INFINITY;
        const RowAt a = row_at(p, row0 + r, h, first, count, len);
        const int64_t flat = a.token * (static_cast<int64_t>(p.cache.kv_heads) * p.group) + a.head;
        if (p.splits > 1) {
            *reinterpret_cast<float4 *>(p.part_o + (flat * p.splits + split) * D + d) = acc;
            if (d == 0)
                p.part_lse[flat * p.splits + split] = lse2;
        } else {
            __nv_bfloat16 *dst =
                static_cast<__nv_bfloat16 *>(p.out.x) + a.token * p.out.token_ld + a.head * p.out.head_ld + d;
            const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x, acc.y), y = __floats2bfloat162_rn(acc.z, acc.w);
            *reinterpret_cast<uint2 *>(dst) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
            if (d == 0 && p.lse)
                p.lse[flat] = kLn2 * lse2;
        }
    }
}

// Joins the parts of the key axis: one warp per (token, query head).
template <int D> __global__ void __launch_bounds__(256) kv_attend_join_kernel(const KvAttendParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t heads = static_cast<int64_t>(p.cache.kv_heads) * p.group;
    const int64_t flat = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    grid_dependency_wait();
    // tokens outside starts[0] .. starts[seqs] belong to no sequence
    const int64_t token = flat / heads;
    if (token >= p.batch.tokens || token < p.batch.starts[0] || token >= p.batch.starts[p.batch.seqs])
        return;
    const float *lse = p.part_lse + flat * p.splits;
    float top = -INFINITY;
    for (int i = lane; i < p.splits; i += 32)
        top = fmaxf(top, lse[i]);
    for (int o = 16; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    float acc[D / 32] = {};
    float den = 0.0f;
    if (top > -INFINITY) {
        for (int i = 0; i < p.splits; ++i) {
            const float w = exp2_approx(lse[i] - top);
            if (w == 0.0f)
                continue;
            den += w;
            const float *src = p.part_o + (flat * p.splits + i) * D + lane * (D / 32);
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                acc[j] = fmaf(w, src[j], acc[j]);
        }
    }
    const float inv = den > 0.0f ? __frcp_rn(den) : 0.0f;
    const int64_t head = flat % heads;
    __nv_bfloat16 *dst =
        static_cast<__nv_bfloat16 *>(p.out.x) + token * p.out.token_ld + head * p.out.head_ld + lane * (D / 32);
#pragma unroll
    for (int j = 0; j < D / 32; j += 2)
        *reinterpret_cast<__nv_bfloat162 *>(dst + j) = __floats2bfloat162_rn(acc[j] * inv, acc[j + 1] * inv);
    if (p.lse && lane == 0)
        p.lse[flat] = den > 0.0f ? kLn2 * (top + log2f(den)) : -INFINITY;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

cudaError_t launch(const void *k, int64_t grid, int threads, const KvAttendParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    KvAttendParams pp = p;
    void *args[1] = {&pp};
    return cudaLaunchKernelExC(&cfg, k, args);
}

// Up to 16 rows per (sequence, KV head) go to the kernel above, in tiles of 8
// or 16; more rows to the tensor-memory kernel in tiles of 256.
bool narrow(const KvAttendParams &p) { return p.batch.max_new * p.group <= 8; }
bool wide(const KvAttendParams &p) { return p.batch.max_new * p.group > 16; }

template <int D, bool FP8> const void *rows_kernel(bool one)
{
    return one ? reinterpret_cast<const void *>(kv_attend_rows_kernel<D, FP8, 1, 8>)
               : reinterpret_cast<const void *>(kv_attend_rows_kernel<D, FP8, 2, 4>);
}

} // namespace

void kv_attend_plan(KvAttendParams *p)
{
    const int64_t rows = p->batch.max_new * p->group;
    const int64_t len = p->batch.max_len > 0 ? p->batch.max_len : 1;
    const int64_t tile = wide(*p) ? kTileRows : narrow(*p) ? 8 : 16;
    p->row_tiles = static_cast<int32_t>(ceil_div(rows, tile));
    const int64_t ctas = p->batch.seqs * p->cache.kv_heads * p->row_tiles;
    // parts of the key axis: enough CTAs to fill the SMs, each with a few steps
    const int64_t step = narrow(*p) || wide(*p) ? 128 : 64;
    int64_t splits = ctas > 0 ? 148 * (wide(*p) ? 1 : 4) / ctas : 1;
    const int64_t most = ceil_div(len, 2 * step);
    splits = splits > most ? most : splits;
    splits = splits < 1 ? 1 : splits;
    p->split_keys = static_cast<int32_t>(ceil_div(ceil_div(len, splits), step) * step);
    p->splits = static_cast<int32_t>(ceil_div(len, p->split_keys));
}

cudaError_t launch_kv_attend(const KvAttendParams &p, cudaStream_t stream)
{
    cudaError_t e;
    if (wide(p)) {
        e = launch_kv_attend_tiles(p, stream);
    } else {
        const bool one = narrow(p);
        const void *k = p.cache.d == 128 ? (p.cache.fp8 ? rows_kernel<128, true>(one) : rows_kernel<128, false>(one))
                                         : (p.cache.fp8 ? rows_kernel<64, true>(one) : rows_kernel<64, false>(one));
        e = launch(k, p.batch.seqs * p.cache.kv_heads * p.row_tiles * p.splits, one ? 256 : 128, p, stream);
    }
    if (e != cudaSuccess || p.splits <= 1)
        return e;
    const void *join = p.cache.d == 128 ? reinterpret_cast<const void *>(kv_attend_join_kernel<128>)
                                        : reinterpret_cast<const void *>(kv_attend_join_kernel<64>);
    return launch(join, ceil_div(p.batch.tokens * p.cache.kv_heads * p.group, 8), 256, p, stream);
}

} // namespace ss24
