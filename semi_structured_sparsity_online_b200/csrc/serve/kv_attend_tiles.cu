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
//   8         one lane issues the MMAs: S (K-major operands) and O += P V with
//             P in tensor memory and V as it lies (MN-major)
//   9-15      codes of K and V from the pages to fp16 in shared memory, a ring
//             of stages in the 128-byte swizzle that the MMA reads
// The two row tiles take turns: while one warpgroup works on its S, the
// tensor cores serve the other. A new S overwrites the weights of the step
// before; MMAs of one thread run in order, and the commit behind S(j + 1) also
// tells that P V of step j is done, so the output may be rescaled then. That
// happens only when a row's bound M moves by more than 2^8.
#include "kv_attend.cuh"
#include "tcgen05.cuh"

namespace ss24 {

namespace {

constexpr int kTileThreads = 512;
// 512 threads start with 128 registers each; 2 x 128 x (176 + 80) is the same sum
constexpr int kRegsRows = 176, kRegsRest = 80;
constexpr int kKeys = 128;   // keys per step
constexpr int kConvWarps = 7;
constexpr int kRing = 4;     // fp16 stages: K and V of a step take one each
constexpr int kRaw = 2;      // stages of codes on their way from the pages
constexpr int kScaleRing = 4; // steps of page scales

template <int D> struct TileShape {
    static constexpr uint32_t kStage = kKeys * D * 2; // also a row tile of q
    static constexpr uint32_t kAtom = kKeys * 128;    // 128 rows x 128 bytes
    static constexpr uint32_t kCodes = kKeys * D;     // a stage's codes
    static constexpr uint32_t kTiles = (2 + kRing) * kStage + kRaw * kCodes;
    static constexpr size_t kSmem = 1024 + kTiles + kScaleRing * 8 * 16 + 256;
    static_assert(kSmem <= 232448, "shared memory per CTA");
};

constexpr uint32_t kCols = 512; // S0 0, S1 128, O0 256, O1 384
__host__ __device__ constexpr uint32_t f16_idesc(int n, bool b_mn)
{
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

template <int N> __device__ __forceinline__ void regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;"
        : "=f"(r)
        : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return r;
}

struct Bars {
    uint64_t kv_full[kRing], kv_empty[kRing], q_full[2], s_full[2], p_half[2], p_full[2], o_full[2];
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
    float4 *scales = reinterpret_cast<float4 *>(gen + S::kTiles); // [kScaleRing][8]: s_k, log2 s_v, 1 / s_v
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
            mbar_init(&bars->kv_full[i], 32 * kConvWarps);
            mbar_init(&bars->kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 128);
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_half[i], 128);
            mbar_init(&bars->p_full[i], 128);
            mbar_init(&bars->o_full[i], 1);
        }
        fence_barrier_init();
    }
    if (warp == 8)
        tc::alloc(tmem_base, kCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_base;
    bool failed = false;

    if (warp < 8) {
        // ---- a row per thread -------------------------------------------------
        regs_up<kRegsRows>();
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
            // never 0 (a page of zero keys, scale 0): 0 times a masked -infinity is NaN
            auto factor = [&](float s_k) { return fmaxf(s_k * fac, 0x1p-126f); };
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
                uint32_t v[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tc::ld32(ts + 32 * c, v[c]);
                tc::wait_ld();
                if (edge) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (key0 + 32 * c + i >= limit)
                                v[c][i] = 0xff800000u; // -infinity
                }
                float mx = -INFINITY;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const uint32_t *y = &v[g >> 1][16 * (g & 1)];
                    float x = max3(y[0], y[1], y[2]), z = max3(y[3], y[4], y[5]);
                    x = max3(__float_as_uint(x), y[6], y[7]), z = max3(__float_as_uint(z), y[8], y[9]);
                    x = max3(__float_as_uint(x), y[10], y[11]), z = max3(__float_as_uint(z), y[12], y[13]);
                    x = fmaxf(max3(__float_as_uint(x), y[14], y[15]), z);
                    mx = fmaxf(mx, fmaf(x, factor(sc[g].x), sc[g].y));
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
                    uint32_t pk[16];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float4 f = sc[2 * c + g];
                        const float af = factor(f.x), bm = f.y - m;
                        const f32x2 af2 = pack2(af, af), bm2 = pack2(bm, bm);
                        f32x2 sum = pack2(0.0f, 0.0f);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const f32x2 x = fma2(
                                pack2(__uint_as_float(v[c][16 * g + i]), __uint_as_float(v[c][16 * g + i + 1])), af2, bm2);
                            const float x0 = exp2_approx(lo2(x)), x1 = exp2_approx(hi2(x));
                            sum = add2(sum, pack2(x0, x1));
                            pk[8 * g + i / 2] = pack_f16(x0, x1);
                        }
                        l = fmaf(lo2(sum) + hi2(sum), f.z, l);
                    }
                    tc::st16(ts + 16 * c, pk);
                    if (c & 1) {
                        // half of the step's weights: its products may start
                        tc::wait_st();
                        tc::fence_before();
                        mbar_arrive(c == 1 ? &bars->p_half[w] : &bars->p_full[w]);
                    }
                }
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
    } else if (warp > 8) {
        // ---- codes to fp16 ------------------------------------------------------
        regs_down<kRegsRest>();
        constexpr int CPR = D / 16;            // 16-code chunks per key
        constexpr int RPW = 32 / CPR;          // keys a warp takes at a time
        constexpr int GROUPS = kKeys / RPW;    // D = 128: 32 groups of 4 keys; D = 64: 16 of 8
        constexpr int ITERS = (GROUPS + kConvWarps - 1) / kConvWarps;
        const int cw = warp - 9, kr = lane / CPR, cc = lane % CPR;
        const int32_t *table = p.batch.table + s * p.batch.table_ld;
        const int items = 2 * steps;
        const uint32_t raw = skv + kRing * S::kStage + 16 * lane;
        // Group g of this warp's iteration; beyond the last group there is none.
        auto group = [&](int it) { return it * kConvWarps + cw; };
        auto page_at = [&](int32_t key) { return key < ke ? __ldg(table + (key >> p.cache.log2_page)) : -2; };
        auto checked = [&](int32_t id) { // -2: no keys there
            if (id >= p.cache.pages || id == -1 || id < -2) {
                atomicCAS(p.err, 0, kErrPage);
                return -2;
            }
            return id;
        };
        // Codes travel by asynchronous copies, kRaw items ahead; a thread reads
        // back only what it copied itself. Keys past the end and pages outside
        // the cache are zeros. A step's page numbers are loaded a step before
        // they are used; its K and V share the offsets.
        int64_t at[ITERS]; // byte offset of this thread's codes, -1: none
        int32_t next_ids[ITERS];
        auto load_ids = [&](int j) {
#pragma unroll
            for (int it = 0; it < ITERS; ++it)
                next_ids[it] = group(it) < GROUPS
                                   ? page_at(static_cast<int32_t>(kb) + j * kKeys + group(it) * RPW + kr) : -2;
        };
        auto fetch = [&](int item) {
            if (item < items) {
                if ((item & 1) == 0) {
                    const int32_t key0 = static_cast<int32_t>(kb) + (item >> 1) * kKeys + kr;
#pragma unroll
                    for (int it = 0; it < ITERS; ++it) {
                        const int32_t id = checked(next_ids[it]);
                        const int32_t slot = (key0 + group(it) * RPW) & (p.cache.page - 1);
                        at[it] = id < 0 ? -1 : (((static_cast<int64_t>(id) * p.cache.kv_heads + h) << p.cache.log2_page) +
                                                slot) * D + 16 * cc;
                    }
                    load_ids((item >> 1) + 1);
                }
                const uint8_t *codes = p.cache.codes[item & 1];
#pragma unroll
                for (int it = 0; it < ITERS; ++it)
                    if (group(it) < GROUPS)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                         raw + (item % kRaw) * S::kCodes + group(it) * 512),
                                     "l"(codes + (at[it] < 0 ? 0 : at[it])), "r"(at[it] < 0 ? 0 : 16));
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // s_k and s_v of 16-key group `lane` of a step (lanes 0-7 of the first
        // warp), a step ahead; s_v < 0: no keys
        const bool scaler = cw == 0 && lane < 8;
        float s_k = 0.0f, s_v = -1.0f;
        int32_t scale_id = -2;
        auto load_scale_id = [&](int j) {
            if (scaler)
                scale_id = page_at(static_cast<int32_t>(kb) + j * kKeys + 16 * lane);
        };
        auto load_scales = [&] {
            const bool on = scale_id >= 0 && scale_id < p.cache.pages;
            const int64_t ph = on ? static_cast<int64_t>(scale_id) * p.cache.kv_heads + h : 0;
            s_k = on ? __ldg(p.cache.scales[0] + ph) : 0.0f;
            s_v = on ? __ldg(p.cache.scales[1] + ph) : -1.0f;
        };
        load_ids(0);
        load_scale_id(0);
        load_scales();
        load_scale_id(1);
        for (int item = 0; item < kRaw; ++item)
            fetch(item);
        for (int item = 0; item < items; ++item) {
            const int st = item % kRing;
            if (item >= kRing && !mbar_wait(&bars->kv_empty[st], (item / kRing - 1) & 1, p.wait_limit_ns)) {
                failed = true;
                break;
            }
            asm volatile("cp.async.wait_group %0;" ::"n"(kRaw - 1) : "memory");
            const uint32_t dst = skv + st * S::kStage;
            uint32_t u[ITERS][4];
#pragma unroll
            for (int it = 0; it < ITERS; ++it)
                if (group(it) < GROUPS)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(u[it][0]), "=r"(u[it][1]), "=r"(u[it][2]), "=r"(u[it][3])
                                 : "r"(raw + (item % kRaw) * S::kCodes + group(it) * 512));
#pragma unroll
            for (int it = 0; it < ITERS; ++it) {
                uint32_t f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    codes4_to_f16<FP8>(u[it][i], f[2 * i], f[2 * i + 1]);
                // the second half of a row's lanes swaps its two stores: all 8 lanes of a
                // store phase then hit different banks
                const int r = group(it) * RPW + kr;
                const bool odd = (cc & 4) != 0;
                const uint32_t a0 = dst + chunk_at<D>(r, 2 * cc), a1 = a0 ^ 16;
                if (group(it) < GROUPS) {
                    sts16(odd ? a1 : a0, odd ? f[4] : f[0], odd ? f[5] : f[1], odd ? f[6] : f[2], odd ? f[7] : f[3]);
                    sts16(odd ? a0 : a1, odd ? f[0] : f[4], odd ? f[1] : f[5], odd ? f[2] : f[6], odd ? f[3] : f[7]);
                }
            }
            if ((item & 1) == 0 && scaler) {
                // with a step's K, the scales of its 16-key groups
                const float sv = fmaxf(s_v, 0x1p-100f);
                scales[(item / 2 % kScaleRing) * 8 + lane] =
                    s_v < 0.0f ? make_float4(0.0f, -INFINITY, 0.0f, 0.0f)
                               : make_float4(s_k, log2f(sv), __frcp_rn(sv), 0.0f);
            }
            tc::fence_proxy();
            mbar_arrive(&bars->kv_full[st]);
            if ((item & 1) == 0 && scaler) {
                load_scales();
                load_scale_id((item >> 1) + 2);
            }
            fetch(item + kRaw);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        regs_down<kRegsRest>();
        if (lane == 0 && steps > 0) {
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
        // the first or second half of a step's keys
        auto values = [&](int w, int st, int j, int half) {
            const uint32_t v = skv + st * S::kStage;
#pragma unroll
            for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
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
                if (!wait(&bars->p_half[w], j & 1))
                    break;
                tc::fence_after();
                values(w, vs, j, 0);
                if (!wait(&bars->p_full[w], j & 1))
                    break;
                tc::fence_after();
                values(w, vs, j, 1);
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
    }
    if (failed)
        atomicCAS(p.err, 0, kErrAttendWait);
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 8) {
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
