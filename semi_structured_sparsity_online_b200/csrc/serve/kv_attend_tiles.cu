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
//   8, 9      one lane each issues a row tile's MMAs: S (K-major operands) and
//             O += P V with P in tensor memory and V as it lies (MN-major). An MMA
//             takes some ten instructions to issue, 70 - 85 cycles between the other
//             warps' of its scheduler, as long as it runs: hence two warps.
//   10-15     codes of K and V from the pages to fp16 in shared memory, a ring
//             of stages in the 128-byte swizzle that the MMA reads
//
// PAIR: two CTAs of a cluster work on twice the rows with cta_group::2 MMAs.
// Each brings half of every B operand (64 keys of K, 64 of the 128 elements of
// V) and its own rows: conversion and the shared-memory reads of K and V halve
// per SM. (Per step of 128 keys the single form converts 32 KB of codes and
// moves 320 KB through shared memory, 2500 cycles beside 2048 of MMA.) The even
// CTA's lanes issue for both; barriers that they wait on are arrived on by both.
//
// A step's S is handled in two halves of 64 keys with barriers of their own:
// while a row's thread works on one half, the tensor cores multiply the weights
// of the other with V and form the next S in its place (MMAs of one thread run
// in order, so a new S may overwrite the weights that the MMA before it read).
// In whole steps a row tile's softmax and its MMAs waited for each other, 2400
// and 1400 cycles of a step of 4100. The output is rescaled when a row's bound M
// moves by more than 2^8, which waits for the other half's products first.
//
// Measured: a prompt of 8192 tokens, 32 heads of 128 on 8 KV heads, INT8, pages of
// 64: 544 - 565 us, 1.0 PFLOP/s (0.61 of the measured peak), tensor pipe 48% and
// special-function unit 48% active. 4 x up to 509 tokens over up to 4000 keys, 28
// heads of 64 on 4, E4M3, pages of 16: 82 - 86 us, special functions 52%.
#include "kv_attend.cuh"
#include "tcgen05.cuh"

namespace ss24 {

namespace {

constexpr int kTileThreads = 512;
// 512 threads start with 128 registers each; 2 x 128 x (176 + 80) is the same sum
constexpr int kRegsRows = 176, kRegsRest = 80;
constexpr int kKeys = 128;   // keys per step
constexpr int kConvWarps = 6;

template <int D, bool PAIR> struct TileShape {
    static constexpr int kKRows = PAIR ? kKeys / 2 : kKeys; // keys of K in this CTA
    static constexpr int kVCols = PAIR ? D / 2 : D;         // elements of V in this CTA
    static constexpr int kRing = PAIR ? 8 : 4;              // fp16 stages: K and V of a step take one each
    static constexpr int kRaw = PAIR ? 4 : 2;               // stages of codes on their way from the pages
    static constexpr int kScaleRing = kRing / 2 + 2;        // steps of page scales
    static constexpr uint32_t kQ = 128 * D * 2;             // a row tile of q
    static constexpr uint32_t kStage = kKRows * D * 2;      // equals kKeys * kVCols * 2
    static constexpr uint32_t kQAtom = 128 * 128, kKAtom = kKRows * 128, kVAtom = kKeys * 128; // 128-byte columns
    static constexpr uint32_t kCodes = kKRows * D;          // a stage's codes
    static constexpr uint32_t kTiles = 2 * kQ + kRing * kStage + kRaw * kCodes;
    static constexpr size_t kSmem = 1024 + kTiles + kScaleRing * 8 * 16 + 512;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static_assert(!PAIR || D == 128, "half of V's columns fill a swizzle row");
};

constexpr uint32_t kCols = 512; // S0 0, S1 128, O0 256, O1 384
__host__ __device__ constexpr uint32_t f16_idesc(int m, int n, bool b_mn)
{
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
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

constexpr int kMaxRing = 8;
struct Bars {
    uint64_t kv_full[kMaxRing], kv_empty[kMaxRing], q_full[2], s_full[2][2], p_full[2][2], o_full[2];
};

// 16-byte chunk c (8 fp16) of row r in swizzled atoms of 128 bytes a row.
__device__ __forceinline__ uint32_t chunk_at(uint32_t atom, int r, int c)
{
    return (c >> 3) * atom + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Key n of half h of a step, and V's first row of k step ks of it. A pair's CTAs
// bring 32 of a half's keys each: of keys 0-63 of the step and of keys 64-127.
template <bool PAIR> __device__ __forceinline__ constexpr int half_key(int h, int n)
{
    return PAIR ? (n < 32 ? 32 * h + n : 64 + 32 * h + (n - 32)) : 64 * h + n;
}

// COARSE: pages of 32 or more, so that 32 neighbouring keys share their scales.
template <int D, bool FP8, bool PAIR, bool COARSE>
__global__ void __launch_bounds__(kTileThreads, 1) kv_attend_tiles_kernel(const KvAttendParams p)
{
    using S = TileShape<D, PAIR>;
    constexpr int RING = S::kRing, CTAS = PAIR ? 2 : 1, ROWS = CTAS * kTileRows;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t *gen = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t sq = base, skv = base + 2 * S::kQ;
    float4 *scales = reinterpret_cast<float4 *>(gen + S::kTiles); // [][8]: s_k, log2 s_v, 2^-7 / s_v
    Bars *bars = reinterpret_cast<Bars *>(scales + S::kScaleRing * 8);
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(bars + 1);

    const int tid = threadIdx.x, warp = tc::uniform(tid >> 5), lane = tid & 31;
    const uint32_t rank = PAIR ? tc::cluster_rank() : 0;
    uint32_t b = blockIdx.x / CTAS;
    const int split = b % p.splits;
    b /= p.splits;
    const int h = b % p.cache.kv_heads;
    b /= p.cache.kv_heads;
    // the last row tiles see the most keys: they start first
    const int64_t tile = p.row_tiles - 1 - b % p.row_tiles;
    grid_dependency_wait();
    // where the CTAs are more than the SMs
    const int64_t s = gridDim.x > 148 ? longest_first(p.batch, b / p.row_tiles, reinterpret_cast<int32_t *>(gen))
                                      : b / p.row_tiles;

    int32_t first, count, len;
    const bool known = kv_sequence(p.batch, s, p.err, &first, &count, &len);
    const int64_t row0 = tile * ROWS, rows = static_cast<int64_t>(count) * p.group;
    if (!known || row0 >= rows)
        return;
    // MMA row tile w holds rows 128 CTAS w on; the CTA of rank r its r-th 128
    const int live = static_cast<int>(rows - row0 < ROWS ? rows - row0 : ROWS);
    const bool two = tc::uniform(live > 128 * CTAS);
    const int64_t kb = static_cast<int64_t>(split) * p.split_keys;
    int64_t ke = kb + p.split_keys;
    const int32_t last = row_at(p, row0 + live - 1, h, first, count, len).limit;
    if (ke > last)
        ke = last;
    const int steps = tc::uniform(ke > kb ? static_cast<int>((ke - kb + kKeys - 1) / kKeys) : 0);

    if (tid == 0) {
        // arrivals come from warps, of both CTAs
        for (int i = 0; i < RING; ++i) {
            mbar_init(&bars->kv_full[i], CTAS * kConvWarps);
            mbar_init(&bars->kv_empty[i], two ? 2 : 1); // from the issuing warps
        }
        for (int i = 0; i < 2; ++i) {
            // warps that have rows of row tile i
            const int warps = (live - 128 * CTAS * i + 31) / 32;
            mbar_init(&bars->q_full[i], CTAS * 4);
            for (int half = 0; half < 2; ++half) {
                mbar_init(&bars->s_full[i][half], 1);
                mbar_init(&bars->p_full[i][half], warps < 1 ? 1 : warps < 4 * CTAS ? warps : 4 * CTAS);
            }
            mbar_init(&bars->o_full[i], 1);
        }
        fence_barrier_init();
    }
    if (warp == 8) {
        if constexpr (PAIR)
            tc::alloc_pair(tmem_base, kCols);
        else
            tc::alloc(tmem_base, kCols);
    }
    tc::fence_before();
    __syncthreads();
    if constexpr (PAIR)
        tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = tc::uniform(*tmem_base);
    bool failed = false;
    // a warp's arrival on a barrier that the issuing lane waits on
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) {
            if constexpr (PAIR)
                tc::arrive_cluster(tc::cluster_addr(smem_u32(bar), 0));
            else
                mbar_arrive(bar);
        }
    };

    if (warp < 8) {
        // ---- a row per thread -------------------------------------------------
        regs_up<kRegsRows>();
        const int w = warp >> 2, r = tid & 127, row = 128 * (CTAS * w + rank) + r;
        if (w == 0 || two) {
            const bool on = row < live;
            const RowAt a = row_at(p, row0 + (on ? row : 0), h, first, count, len);
            // a row behind the tile's last needs no mask: nothing reads its result (40
            // rows over 16 x 8192 keys, heads of 64: 86 us; masked in every step, and with
            // the warps that have no row at work, 114)
            const int32_t limit = on ? a.limit : INT32_MAX;
            // a warp without rows leaves S as its weights, and is not waited for
            const int halves = __any_sync(kFull, on) ? 2 * steps : 0;
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
                const int e = query_exponent(static_cast<int>(top >> 7) - 127);
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
                    sts16(sq + w * S::kQ + chunk_at(S::kQAtom, r, c), f[0], f[1], f[2], f[3]);
                }
            }
            tc::fence_proxy();
            arrive(&bars->q_full[w]);

            const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
            const uint32_t ts0 = tmem + lanes + 128 * w, to = tmem + lanes + 256 + 128 * w;
            const int32_t low = __reduce_min_sync(kFull, limit);
            // never 0 (a page of zero keys, scale 0): 0 times a masked -infinity is NaN
            auto factor = [&](float s_k) { return fmaxf(s_k * fac, 0x1p-126f); };
            constexpr int GS = COARSE ? 32 : 16, GN = 64 / GS; // keys that share scales, such groups
            float m = -1e30f, top = -1e30f, l = 0.0f;
            for (int i = 0; i < halves; ++i) {
                const int j = i >> 1, half = i & 1;
                // a lane that gives up says so in the vote below
                const bool late = !tc::wait(&bars->s_full[w][half], j & 1, p.wait_limit_ns);
                tc::fence_after();
                const uint32_t ts = ts0 + 64 * half; // S, and the weights in its first half
                const int32_t key0 = static_cast<int32_t>(kb) + j * kKeys;
                const float4 *sc = scales + (j % S::kScaleRing) * 8;
                uint32_t v[64];
                __syncwarp();
                tc::ld32(ts, reinterpret_cast<uint32_t(&)[32]>(v[0]));
                tc::ld32(ts + 32, reinterpret_cast<uint32_t(&)[32]>(v[32]));
                tc::wait_ld();
                if (key0 + kKeys > low) {
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (key0 + half_key<PAIR>(half, k) >= limit)
                            v[k] = 0xff800000u; // -infinity
                }
                float4 f[GN];
#pragma unroll
                for (int g = 0; g < GN; ++g) {
                    f[g] = sc[half_key<PAIR>(half, GS * g) >> 4];
                    f[g].x = factor(f[g].x);
                }
                // the largest exponent in the row's 64 keys
                float mx = -INFINITY;
#pragma unroll
                for (int g = 0; g < GN; ++g) {
                    const uint32_t *y = v + GS * g;
                    float x = max3(y[0], y[1], y[2]), z = max3(y[3], y[4], y[5]);
#pragma unroll
                    for (int k = 6; k + 3 < GS; k += 4) {
                        x = max3(__float_as_uint(x), y[k], y[k + 1]);
                        z = max3(__float_as_uint(z), y[k + 2], y[k + 3]);
                    }
                    x = max3(__float_as_uint(x), y[GS - 2], y[GS - 1]);
                    mx = fmaxf(mx, fmaf(fmaxf(x, z), f[g].x, f[g].y));
                }
                if (__any_sync(kFull, late || weight_off(m, mx))) {
                    if (__any_sync(kFull, late)) {
                        failed = true;
                        break;
                    }
                    const float mn = weight_reference(m, mx, top, l < kFallBelow), scale = exp2_approx(m - mn);
                    const bool moved = __any_sync(kFull, mn != m);
                    m = mn;
                    top = fmaxf(top, mn);
                    l *= scale;
                    if (i > 0 && moved) {
                        // the half before: its products are done when the S behind them is (or,
                        // in the last step, when the barrier that stands for it says so)
                        if (!tc::wait_warp(&bars->s_full[w][half ^ 1], (j + half) & 1, p.wait_limit_ns)) {
                            failed = true;
                            break;
                        }
                        tc::fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tc::ld32(to + c, o);
                            tc::wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * scale);
                            tc::st32(to + c, o);
                        }
                        tc::wait_st();
                    }
                }
                // the weights, in pairs over v[0 .. 31]; their sum over the V scales
#pragma unroll
                for (int g = 0; g < GN; ++g) {
                    const float bm = f[g].y - m;
                    const f32x2 af2 = pack2(f[g].x, f[g].x), bm2 = pack2(bm, bm);
                    f32x2 sum = pack2(0.0f, 0.0f);
#pragma unroll
                    for (int k = GS * g; k < GS * g + GS; k += 2) {
                        const f32x2 x = fma2(pack2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), af2, bm2);
                        const f32x2 e = pack2(exp2_approx(lo2(x)), exp2_approx(hi2(x)));
                        sum = add2(sum, e);
                        v[k / 2] = pack_f16(lo2(e), hi2(e));
                    }
                    l = fmaf(lo2(sum) + hi2(sum), f[g].z, l);
                }
                tc::st32(ts, reinterpret_cast<uint32_t(&)[32]>(v[0]));
                tc::wait_st();
                tc::fence_before();
                arrive(&bars->p_full[w][half]);
            }

            // ---- the row's output -------------------------------------------------
            // also after a wait that ran out: the commit's arrival comes before the CTA exits
            if (steps > 0 && !tc::wait_warp(&bars->o_full[w], 0, p.wait_limit_ns))
                failed = true;
            tc::fence_after();
            const bool any = steps > 0 && l != 0.0f; // NaN from a NaN in q
            const float inv = any ? weight_inverse(l) : 0.0f;
            const float lse2 = any ? m + kWeightUnitLog + log2f(l) : -INFINITY;
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
    } else if (warp > 9) {
        // ---- codes to fp16 ------------------------------------------------------
        regs_down<kRegsRest>();
        // Of K and of V: 16-code chunks per key in this CTA, keys a warp takes at a
        // time, groups of those
        constexpr int CPR[2] = {D / 16, S::kVCols / 16};
        constexpr int RPW[2] = {32 / CPR[0], 32 / CPR[1]};
        constexpr int GROUPS = S::kKRows / RPW[0]; // the same for V
        constexpr int ITERS = PAIR ? (GROUPS + kConvWarps - 1) / kConvWarps : GROUPS / 4;
        static_assert(PAIR || GROUPS % 8 == 0, "groups for four and for eight warps");
        constexpr int AHEAD = S::kRaw / 2;
        static_assert(kKeys / RPW[1] == GROUPS, "K and V items have one size");
        const int cw = warp - 10;
        // A lane's key and chunk: 8 neighbouring lanes write 4 chunks of two
        // neighbouring rows, whose swizzled places fall on different banks.
        int kr[2], cc[2];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            kr[kv] = CPR[kv] == 8 ? (lane >> 2) & 3 : lane >> 2;
            cc[kv] = CPR[kv] == 8 ? (lane & 3) + (lane >> 4 << 2) : lane & 3;
        }
        const int32_t *table = p.batch.table + s * p.batch.table_ld;
        const uint32_t raw = skv + RING * S::kStage + 16 * lane;
        const int32_t end = static_cast<int32_t>(ke), begin = static_cast<int32_t>(kb);
        // This warp's group in an iteration; beyond the last group there is none. A pair's
        // warps take equal shares. A single CTA converts twice as much per step: every
        // scheduler of the SM takes a quarter, two with one of these warps, two with two
        // (240 rows over 16 x 8192 keys, heads of 128: 157 us, in equal shares 166; 480
        // rows in pairs 278 and 274).
        const int sch = warp & 3;
        const int stride = PAIR ? kConvWarps : sch < 2 ? 4 : 8, start = PAIR ? cw : sch + (warp >= 14 ? 4 : 0);
        auto group = [&](int it) { return it * stride + start; };
        // Items come in the order K0, K1, V0, K2, V1, ...: when V of a step is there,
        // K of the next is too, and the issuing lane waits once for both.
        auto raw_at = [&](int j, int kv) {
            const int n = kv == 1 ? 2 * j + 2 : j > 0 ? 2 * j - 1 : 0;
            return raw + (n & (S::kRaw - 1)) * S::kCodes;
        };
        // Lanes 0-7 look up the 16-key groups of a step: the cache row of the
        // group's first key (-1: no keys), and for the first warp its scales. Page
        // numbers are loaded a step ahead; the scales of the step before go to
        // shared memory. K of a step is fetched before V of the step before it.
        auto load_id = [&](int j) {
            const int32_t key = begin + j * kKeys + 16 * lane;
            return lane < 8 && key < end ? __ldg(table + (key >> p.cache.log2_page)) : -1;
        };
        int32_t id = load_id(0), row = -1, row_before = -1;
        float s_k = 0.0f, s_v = -1.0f; // s_v < 0: no keys
        auto next_rows = [&](int j) {
            if (cw == 0 && lane < 8 && j > 0) {
                const float sv = fmaxf(s_v, 0x1p-100f);
                scales[((j - 1) % S::kScaleRing) * 8 + lane] =
                    s_v < 0.0f ? make_float4(0.0f, -INFINITY, 0.0f, 0.0f)
                               : make_float4(s_k, log2f(sv), __frcp_rn(sv) * kWeightUnit, 0.0f);
            }
            const int32_t key = begin + j * kKeys + 16 * lane;
            const bool there = lane < 8 && key < end, on = there && id >= 0 && id < p.cache.pages;
            if (there && !on)
                atomicCAS(p.err, 0, kErrPage);
            const int32_t ph = on ? id * p.cache.kv_heads + h : 0;
            row_before = row;
            row = on ? (ph << p.cache.log2_page) + (key & (p.cache.page - 1)) : -1;
            if (cw == 0) {
                s_k = on ? __ldg(p.cache.scales[0] + ph) : 0.0f;
                s_v = on ? __ldg(p.cache.scales[1] + ph) : -1.0f;
            }
            id = load_id(j + 1);
        };
        // Codes travel by asynchronous copies, kRaw items ahead; a thread reads
        // back only what it copied itself. Keys past the end and pages outside
        // the cache are zeros.
        auto fetch = [&](int j, int kv) {
            if (j < steps) {
                const uint8_t *codes = p.cache.codes[kv] + 16 * cc[kv] + (kv == 1 ? rank * S::kVCols : 0);
#pragma unroll
                for (int it = 0; it < ITERS; ++it) {
                    // the key's place in the step
                    const int32_t at = (kv == 0 ? static_cast<int32_t>(rank) * S::kKRows : 0) + group(it) * RPW[kv] + kr[kv];
                    if (group(it) >= GROUPS)
                        break;
                    const int32_t first_row = __shfl_sync(kFull, kv == 0 ? row : row_before, at >> 4);
                    const bool on = first_row >= 0 && begin + j * kKeys + at < end;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(raw_at(j, kv) + group(it) * 512),
                                 "l"(on ? codes + static_cast<int64_t>(first_row + (at & 15)) * D
                                        : static_cast<const uint8_t *>(p.q.x)), // nothing is read there
                                 "r"(on ? 16 : 0));
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // One item: the codes at src to fp16 in the stage at dst.
        auto convert = [&](uint32_t src, uint32_t dst, int kv) {
            uint32_t u[ITERS][4];
#pragma unroll
            for (int it = 0; it < ITERS; ++it)
                if (group(it) < GROUPS)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(u[it][0]), "=r"(u[it][1]), "=r"(u[it][2]), "=r"(u[it][3])
                                 : "r"(src + group(it) * 512));
#pragma unroll
            for (int it = 0; it < ITERS; ++it) {
                uint32_t f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    codes4_to_f16<FP8>(u[it][i], f[2 * i], f[2 * i + 1]);
                const uint32_t a = dst + chunk_at(kv == 0 ? S::kKAtom : S::kVAtom, group(it) * RPW[kv] + kr[kv], 2 * cc[kv]);
                if (group(it) < GROUPS) {
                    sts16(a, f[0], f[1], f[2], f[3]);
                    sts16(a ^ 16, f[4], f[5], f[6], f[7]);
                }
            }
        };
        next_rows(0);
        fetch(0, 0);
        next_rows(1);
        fetch(1, 0);
        if constexpr (AHEAD == 2) {
            fetch(0, 1);
            next_rows(2);
            fetch(2, 0);
        }
        int st = 0, phase = 1;
        for (int i = 0; i <= steps && !failed; ++i) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) { // K of step i, V of step i - 1
                const int j = i - kv;
                if (j < 0 || j >= steps)
                    continue;
                if (!tc::wait_warp(&bars->kv_empty[st], phase, p.wait_limit_ns)) {
                    failed = true;
                    break;
                }
                // the last V has no K between it and the V before
                if (kv == 1 && i == steps)
                    asm volatile("cp.async.wait_group %0;" ::"n"(S::kRaw - 2) : "memory");
                else
                    asm volatile("cp.async.wait_group %0;" ::"n"(S::kRaw - 1) : "memory");
                if (kv == 0 && j > 0)
                    next_rows(j + AHEAD);
                convert(raw_at(j, kv), skv + st * S::kStage, kv);
                tc::fence_proxy();
                if (kv == 0 || j != p.test_skip || blockIdx.x != 0 || cw != 0)
                    arrive(&bars->kv_full[st]);
                // the item kRaw on takes the slot
                if (kv == 0 && j == 0)
                    fetch(AHEAD - 1, 1);
                else
                    fetch(j + AHEAD, kv);
                if (++st == RING)
                    st = 0, phase ^= 1;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        regs_down<kRegsRest>();
        const int w = warp - 8;
        if (w < (two ? 2 : 1) && rank == 0 && steps > 0) {
            const bool lead = lane == 0;
            // ---- MMAs -----------------------------------------------------------
            constexpr uint32_t kIS = f16_idesc(128 * CTAS, kKeys / 2, false), kIO = f16_idesc(128 * CTAS, D, true);
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                const bool ok = tc::wait(bar, parity, p.wait_limit_ns);
                tc::fence_after();
                failed = __any_sync(kFull, !ok);
                return !failed;
            };
            auto commit = [&](uint64_t *bar) {
                if constexpr (PAIR)
                    tc::commit_pair(bar, lead);
                else
                    tc::commit(bar, lead);
            };
            const uint32_t q_low = tc::desc_low_kmajor(sq), k_low = tc::desc_low_kmajor(skv);
            const uint32_t v_low = tc::desc_low_mnmajor(skv, S::kVAtom);
            // S of one half of a step's keys: K rows 64 half (of a pair 32 half in each CTA)
            auto scores = [&](int st, int half) {
                const uint32_t q = q_low + w * (S::kQ >> 4), k = k_low + (st * S::kStage + half * (S::kKAtom / 2) >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint64_t a = tc::desc(q + (ks >> 2) * (S::kQAtom >> 4) + (ks & 3) * 2);
                    const uint64_t b = tc::desc(k + (ks >> 2) * (S::kKAtom >> 4) + (ks & 3) * 2);
                    if constexpr (PAIR)
                        tc::mma_f16_pair(tmem + 128 * w + 64 * half, a, b, kIS, ks > 0, lead);
                    else
                        tc::mma_f16(tmem + 128 * w + 64 * half, a, b, kIS, ks > 0, lead);
                }
            };
            auto values = [&](int st, int j, int half) {
                const uint32_t v = v_low + st * (S::kStage >> 4);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t b = tc::desc(v + half_key<PAIR>(half, 16 * ks) * (128 >> 4));
                    const uint32_t a = tmem + 128 * w + 64 * half + 8 * ks, d = tmem + 256 + 128 * w;
                    if constexpr (PAIR)
                        tc::mma_f16_ta_pair(d, a, b, kIO, j > 0 || half > 0 || ks > 0, lead);
                    else
                        tc::mma_f16_ta(d, a, b, kIO, j > 0 || half > 0 || ks > 0, lead);
                }
            };
            int next = 0, phase = 0; // the next item's stage
            auto advance = [&] {
                if (++next == RING)
                    next = 0, phase ^= 1;
            };
            bool fine = wait(&bars->q_full[w], 0) && wait(&bars->kv_full[0], 0);
            if (fine) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    scores(0, half);
                    commit(&bars->s_full[w][half]);
                }
                commit(&bars->kv_empty[0]);
            }
            advance();
            for (int j = 0; j < steps && fine; ++j) {
                const bool more = j + 1 < steps;
                const int ks = next;
                if (more)
                    advance();
                const int vs = next;
                fine = wait(&bars->kv_full[vs], phase); // and K before it
                advance();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    fine = fine && wait(&bars->p_full[w][half], j & 1);
                    if (!fine)
                        break;
                    values(vs, j, half);
                    if (more)
                        scores(ks, half);
                    commit(&bars->s_full[w][half]);
                }
                commit(&bars->kv_empty[vs]);
                if (more)
                    commit(&bars->kv_empty[ks]);
            }
            commit(&bars->o_full[w]);
            // every MMA has finished before the tensor memory goes
            (void)tc::wait(&bars->o_full[w], 0, p.wait_limit_ns);
        }
    }
    if (failed)
        atomicCAS(p.err, 0, kErrAttendWait);
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if constexpr (PAIR)
        tc::cluster_sync();
    if (warp == 8) {
        tc::fence_after();
        if constexpr (PAIR)
            tc::dealloc_pair(tmem, kCols);
        else
            tc::dealloc(tmem, kCols);
    }
}

template <int D, bool FP8, bool PAIR, bool COARSE> cudaError_t launch_tiles(const KvAttendParams &p, cudaStream_t stream)
{
    using S = TileShape<D, PAIR>;
    auto kern = kv_attend_tiles_kernel<D, FP8, PAIR, COARSE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((PAIR ? 2 : 1) * p.batch.seqs * p.cache.kv_heads * p.row_tiles * p.splits));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}


template <int D, bool PAIR> cudaError_t launch_tiles(const KvAttendParams &p, cudaStream_t stream)
{
    if (p.cache.page >= 32)
        return p.cache.fp8 ? launch_tiles<D, true, PAIR, true>(p, stream) : launch_tiles<D, false, PAIR, true>(p, stream);
    return p.cache.fp8 ? launch_tiles<D, true, PAIR, false>(p, stream) : launch_tiles<D, false, PAIR, false>(p, stream);
}

} // namespace

cudaError_t launch_kv_attend_tiles(const KvAttendParams &p, cudaStream_t stream)
{
    if (p.cache.d == 64)
        return launch_tiles<64, false>(p, stream);
    return kv_attend_pairs(p) ? launch_tiles<128, true>(p, stream) : launch_tiles<128, false>(p, stream);
}

} // namespace ss24
