// Attention of many query rows over the 8-bit paged cache on the
// 5th-generation tensor cores (the mathematics and the row order are those of
// kv_attend.cu).
//
// A CTA holds two tiles of 128 rows of one (sequence, KV head) and walks over
// 128 keys at a time. Its warps:
//   0-3, 4-7  one warpgroup per row tile: a thread owns a row. It writes q to
//             shared memory in fp16, takes its row of S = q K^T from tensor
//             memory, forms the weights and writes them back as fp16 over S;
//             row maxima and sums need no shuffle
//   8-11      codes of K and V from the pages to fp16 in shared memory, a ring
//             of stages in the 128-byte swizzle that the MMA reads
//   12        one lane issues the MMAs: S (K-major operands) and O += P V with
//             P in tensor memory and V as it lies (MN-major)
// The two row tiles take turns: while one warpgroup works on its S, the
// tensor cores serve the other. A new S overwrites the weights of the step
// before; MMAs of one thread run in order, and the commit behind S(j + 1) also
// tells that P V of step j is done, so the output may be rescaled then. That
// happens only when a row's bound M moves by more than 2^8.
#include "kv_attend.cuh"
#include "tcgen05.cuh"

namespace ss24 {

namespace {

constexpr int kTileThreads = 416;
constexpr int kKeys = 128;   // keys per step
constexpr int kRing = 5;     // stages: K and V of a step take one each
constexpr int kScaleRing = 4; // steps of page scales

template <int D> struct TileShape {
    static constexpr uint32_t kStage = kKeys * D * 2; // also a row tile of q
    static constexpr uint32_t kAtom = kKeys * 128;    // 128 rows x 128 bytes
    static constexpr size_t kSmem = 1024 + (2 + kRing) * kStage + kScaleRing * 8 * 16 + 256;
    static_assert(kSmem <= 232448, "shared memory per CTA");
};

constexpr uint32_t kCols = 512; // S0 0, S1 128, O0 256, O1 384
__host__ __device__ constexpr uint32_t f16_idesc(int n, bool b_mn)
{
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

struct Bars {
    uint64_t kv_full[kRing], kv_empty[kRing], q_full[2], s_full[2], p_full[2], o_full[2];
};

// 16-byte chunk c (8 fp16) of row r in a tile of D / 64 swizzled atoms.
template <int D> __device__ __forceinline__ uint32_t chunk_at(int r, int c)
{
    return (c >> 3) * TileShape<D>::kAtom + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kTileThreads, 1) kv_attend_tiles_kernel(const KvAttendParams p)
{
    using S = TileShape<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t *gen = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t sq = base, skv = base + 2 * S::kStage;
    float4 *scales = reinterpret_cast<float4 *>(gen + (2 + kRing) * S::kStage); // [kScaleRing][8]: s_k, log2 s_v, 1 / s_v
    Bars *bars = reinterpret_cast<Bars *>(scales + kScaleRing * 8);
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(bars + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t b = blockIdx.x;
    const int split = static_cast<int>(b % p.splits);
    b /= p.splits;
    const int h = static_cast<int>(b % p.cache.kv_heads);
    b /= p.cache.kv_heads;
    // the last row tiles see the most keys: they start first
    const int64_t tile = p.row_tiles - 1 - b % p.row_tiles, s = b / p.row_tiles;
    grid_dependency_wait();

    int32_t first, count, len;
    const bool fine = kv_sequence(p.batch, s, p.err, &first, &count, &len);
    const int64_t row0 = tile * kTileRows, rows = static_cast<int64_t>(count) * p.group;
    if (!fine || row0 >= rows)
        return;
    const int live = static_cast<int>(rows - row0 < kTileRows ? rows - row0 : kTileRows);
    const bool two = live > 128;
    const int64_t kb = static_cast<int64_t>(split) * p.split_keys;
    int64_t ke = kb + p.split_keys;
    const int32_t last = row_at(p, row0 + live - 1, h, first, count, len).limit;
    if (ke > last)
        ke = last;
    const int steps = ke > kb ? static_cast<int>((ke - kb + kKeys - 1) / kKeys) : 0;

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&bars->kv_full[i], 128);
            mbar_init(&bars->kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 128);
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i], 128);
            mbar_init(&bars->o_full[i], 1);
        }
        fence_barrier_init();
    }
    if (warp == 12)
        tc::alloc(tmem_base, kCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_base;
    bool failed = false;

    if (warp < 8) {
        // ---- a row per thread -------------------------------------------------
        const int w = warp >> 2, r = tid & 127, row = 128 * w + r;
        if (w == 0 || two) {
            const bool on = row < live;
            const RowAt a = row_at(p, row0 + (on ? row : 0), h, first, count, len);
            const int32_t limit = on ? a.limit : 0;
            float fac = 0.0f;
            {
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q.x) +
                                                                   a.token * p.q.token_ld + a.head * p.q.head_ld);
                uint32_t top = 0; // largest magnitude: bf16 bits order as integers
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = __ldg(src + c);
                    top = max(top, max(max(v.x & 0x7fff, (v.x >> 16) & 0x7fff), max(v.y & 0x7fff, (v.y >> 16) & 0x7fff)));
                    top = max(top, max(max(v.z & 0x7fff, (v.z >> 16) & 0x7fff), max(v.w & 0x7fff, (v.w >> 16) & 0x7fff)));
                }
                int e = static_cast<int>(top >> 7) - 127;
                e = e < -100 ? -100 : e > 100 ? 100 : e;
                // a negative scale turns q, so that the factor of S is never negative
                const float down = on ? copysignf(exp2_int(-e), p.scale_log2) : 0.0f;
                fac = fabsf(p.scale_log2) * exp2_int(e);
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = __ldg(src + c);
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                    uint32_t f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        f[i] = pack_f16(__uint_as_float(u[i] << 16) * down, __uint_as_float(u[i] & 0xffff0000u) * down);
                    sts16(sq + w * S::kStage + chunk_at<D>(r, c), f[0], f[1], f[2], f[3]);
                }
            }
            tc::fence_proxy();
            mbar_arrive(&bars->q_full[w]);

            const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
            const uint32_t ts = tmem + lanes + 128 * w, to = tmem + lanes + 256 + 128 * w;
            const int32_t low = __reduce_min_sync(kFull, limit);
            float m = -1e30f, l = 0.0f;
            for (int j = 0; j < steps; ++j) {
                if (!mbar_wait(&bars->s_full[w], j & 1, p.wait_limit_ns)) {
                    failed = true;
                    break;
                }
                tc::fence_after();
                const int32_t key0 = static_cast<int32_t>(kb) + j * kKeys;
                const bool edge = key0 + kKeys > low;
                const float4 *sc = scales + (j % kScaleRing) * 8;
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    tc::ld32(ts + 32 * c, v);
                    tc::wait_ld();
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float4 f = sc[2 * c + g];
                        float x = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float y = __uint_as_float(v[16 * g + i]);
                            if (edge && key0 + 32 * c + 16 * g + i >= limit)
                                y = -INFINITY;
                            x = fmaxf(x, y);
                        }
                        mx = fmaxf(mx, fmaf(x, f.x * fac, f.y));
                    }
                }
                if (__any_sync(kFull, mx > m + 8.0f)) {
                    const float mn = fmaxf(m, mx), f = exp2_approx(m - mn);
                    m = mn;
                    l *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t v[32];
                            tc::ld32(to + c, v);
                            tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                            tc::st32(to + c, v);
                        }
                        tc::wait_st();
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32], pk[16];
                    tc::ld32(ts + 32 * c, v);
                    tc::wait_ld();
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float4 f = sc[2 * c + g];
                        const float af = f.x * fac, bm = f.y - m;
                        const f32x2 af2 = pack2(af, af), bm2 = pack2(bm, bm);
                        f32x2 sum = pack2(0.0f, 0.0f);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const f32x2 x = fma2(pack2(__uint_as_float(v[16 * g + i]), __uint_as_float(v[16 * g + i + 1])),
                                                 af2, bm2);
                            float x0 = lo2(x), x1 = hi2(x);
                            if (edge) {
                                const int32_t key = key0 + 32 * c + 16 * g + i;
                                x0 = key >= limit ? -INFINITY : x0;
                                x1 = key + 1 >= limit ? -INFINITY : x1;
                            }
                            x0 = exp2_approx(x0);
                            x1 = exp2_approx(x1);
                            sum = add2(sum, pack2(x0, x1));
                            pk[8 * g + i / 2] = pack_f16(x0, x1);
                        }
                        l = fmaf(lo2(sum) + hi2(sum), f.z, l);
                    }
                    tc::st16(ts + 16 * c, pk);
                }
                tc::wait_st();
                tc::fence_before();
                mbar_arrive(&bars->p_full[w]);
            }

            // ---- the row's output -------------------------------------------------
            if (!failed && steps > 0 && !mbar_wait(&bars->o_full[w], 0, p.wait_limit_ns))
                failed = true;
            tc::fence_after();
            const bool any = steps > 0 && l > 0.0f;
            const float inv = any ? __frcp_rn(l) : 0.0f;
            const float lse2 = any ? m + log2f(l) : -INFINITY;
            const int64_t flat = a.token * (static_cast<int64_t>(p.cache.kv_heads) * p.group) + a.head;
            if (!failed) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t v[32];
                    if (steps > 0) {
                        tc::ld32(to + c, v);
                        tc::wait_ld();
                    }
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = any ? __uint_as_float(v[i]) * inv : 0.0f;
                    if (!on)
                        continue;
                    if (p.splits > 1) {
                        float4 *dst = reinterpret_cast<float4 *>(p.part_o + (flat * p.splits + split) * D + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out.x) +
                                                               a.token * p.out.token_ld + a.head * p.out.head_ld + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t u[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const __nv_bfloat162 y = __floats2bfloat162_rn(x[8 * i + 2 * k], x[8 * i + 2 * k + 1]);
                                u[k] = *reinterpret_cast<const uint32_t *>(&y);
                            }
                            dst[i] = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    }
                }
                if (on) {
                    if (p.splits > 1)
                        p.part_lse[flat * p.splits + split] = lse2;
                    else if (p.lse)
                        p.lse[flat] = kLn2 * lse2;
                }
            }
        }
    } else if (warp < 12) {
        // ---- codes to fp16 ------------------------------------------------------
        const int t = tid - 256;
        constexpr int CPR = D / 16;             // 16-code chunks per key
        constexpr int RPI = 128 / CPR;          // keys per iteration
        constexpr int ITERS = kKeys / RPI;      // D = 128: 8 of 16 keys; D = 64: 4 of 32
        const int kr = t / CPR, cc = t % CPR;
        const int32_t *table = p.batch.table + s * p.batch.table_ld;
        const int items = 2 * steps;
        uint4 buf[ITERS];
        auto load = [&](int item) {
            const int32_t key0 = static_cast<int32_t>(kb) + (item >> 1) * kKeys;
#pragma unroll
            for (int it = 0; it < ITERS; ++it) {
                const int32_t key = key0 + it * RPI + kr;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (key < ke) {
                    const int32_t id = __ldg(table + (key >> p.cache.log2_page));
                    if (id >= 0 && id < p.cache.pages) {
                        const int64_t at = (((static_cast<int64_t>(id) * p.cache.kv_heads + h) << p.cache.log2_page) +
                                            (key & (p.cache.page - 1))) * D + 16 * cc;
                        v = __ldg(reinterpret_cast<const uint4 *>(p.cache.codes[item & 1] + at));
                    } else {
                        atomicCAS(p.err, 0, kErrPage);
                    }
                }
                buf[it] = v;
            }
        };
        if (items > 0)
            load(0);
        for (int item = 0; item < items; ++item) {
            const int st = item % kRing;
            if (item >= kRing && !mbar_wait(&bars->kv_empty[st], (item / kRing - 1) & 1, p.wait_limit_ns)) {
                failed = true;
                break;
            }
            const uint32_t dst = skv + st * S::kStage;
#pragma unroll
            for (int it = 0; it < ITERS; ++it) {
                const uint32_t u[4] = {buf[it].x, buf[it].y, buf[it].z, buf[it].w};
                uint32_t f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    codes4_to_f16<FP8>(u[i], f[2 * i], f[2 * i + 1]);
                // the second half of a row's lanes swaps its two stores: all 8 lanes of a
                // store phase then hit different banks
                const int r = it * RPI + kr, odd = (cc >> 2) & 1;
                const uint32_t a0 = dst + chunk_at<D>(r, 2 * cc), a1 = dst + chunk_at<D>(r, 2 * cc + 1);
                if (odd) {
                    sts16(a1, f[4], f[5], f[6], f[7]);
                    sts16(a0, f[0], f[1], f[2], f[3]);
                } else {
                    sts16(a0, f[0], f[1], f[2], f[3]);
                    sts16(a1, f[4], f[5], f[6], f[7]);
                }
            }
            if ((item & 1) == 0 && t < 8) {
                // the scales of the step's 16-key groups, with its K
                const int j = item >> 1;
                const int32_t key = static_cast<int32_t>(kb) + j * kKeys + 16 * t;
                float4 f = make_float4(0.0f, -INFINITY, 0.0f, 0.0f);
                if (key < ke) {
                    const int32_t id = __ldg(table + (key >> p.cache.log2_page));
                    if (id >= 0 && id < p.cache.pages) {
                        const int64_t ph = static_cast<int64_t>(id) * p.cache.kv_heads + h;
                        const float sv = fmaxf(__ldg(p.cache.scales[1] + ph), 0x1p-100f);
                        f = make_float4(__ldg(p.cache.scales[0] + ph), log2f(sv), __frcp_rn(sv), 0.0f);
                    }
                }
                scales[(j % kScaleRing) * 8 + t] = f;
            }
            tc::fence_proxy();
            mbar_arrive(&bars->kv_full[st]);
            if (item + 1 < items)
                load(item + 1);
        }
    } else if (warp == 12 && lane == 0 && steps > 0) {
        // ---- MMAs -----------------------------------------------------------------
        constexpr uint32_t kIS = f16_idesc(kKeys, false), kIO = f16_idesc(D, true);
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!failed && !mbar_wait(bar, parity, p.wait_limit_ns))
                failed = true;
            return !failed;
        };
        auto scores = [&](int w, int st) {
            const uint32_t q = sq + w * S::kStage, k = skv + st * S::kStage;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks >> 2) * S::kAtom + (ks & 3) * 32;
                tc::mma_f16(tmem + 128 * w, tc::desc_kmajor(q + off), tc::desc_kmajor(k + off), kIS, ks > 0);
            }
            tc::commit(&bars->s_full[w]);
        };
        auto values = [&](int w, int st, int j) {
            const uint32_t v = skv + st * S::kStage;
#pragma unroll
            for (int ks = 0; ks < kKeys / 16; ++ks)
                tc::mma_f16_ta(tmem + 256 + 128 * w, tmem + 128 * w + 8 * ks, tc::desc_mnmajor(v + ks * 2048, S::kAtom), kIO,
                               j > 0 || ks > 0);
        };
        const int tiles = two ? 2 : 1;
        for (int w = 0; w < tiles; ++w)
            wait(&bars->q_full[w], 0);
        if (wait(&bars->kv_full[0], 0)) {
            tc::fence_after();
            for (int w = 0; w < tiles; ++w)
                scores(w, 0);
            tc::commit(&bars->kv_empty[0]);
        }
        for (int j = 0; j < steps && !failed; ++j) {
            const int vi = 2 * j + 1, ki = 2 * j + 2, vs = vi % kRing, ks = ki % kRing;
            wait(&bars->kv_full[vs], (vi / kRing) & 1);
            for (int w = 0; w < tiles; ++w) {
                if (!wait(&bars->p_full[w], j & 1))
                    break;
                tc::fence_after();
                values(w, vs, j);
                if (w == tiles - 1)
                    tc::commit(&bars->kv_empty[vs]);
                if (j + 1 < steps) {
                    if (w == 0 && !wait(&bars->kv_full[ks], (ki / kRing) & 1))
                        break;
                    tc::fence_after();
                    scores(w, ks);
                    if (w == tiles - 1)
                        tc::commit(&bars->kv_empty[ks]);
                }
            }
        }
        for (int w = 0; w < 2; ++w)
            tc::commit(&bars->o_full[w]);
        // every MMA has finished before the tensor memory goes
        (void)mbar_wait(&bars->o_full[0], 0, p.wait_limit_ns);
    }
    if (failed)
        atomicCAS(p.err, 0, kErrAttendWait);
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 12) {
        tc::fence_after();
        tc::dealloc(tmem, kCols);
    }
}

} // namespace

cudaError_t launch_kv_attend_tiles(const KvAttendParams &p, cudaStream_t stream)
{
    const bool wide = p.cache.d == 128;
    auto kern = wide ? (p.cache.fp8 ? kv_attend_tiles_kernel<128, true> : kv_attend_tiles_kernel<128, false>)
                     : (p.cache.fp8 ? kv_attend_tiles_kernel<64, true> : kv_attend_tiles_kernel<64, false>);
    const size_t smem = wide ? TileShape<128>::kSmem : TileShape<64>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch.seqs * p.cache.kv_heads * p.row_tiles * p.splits));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

} // namespace ss24
