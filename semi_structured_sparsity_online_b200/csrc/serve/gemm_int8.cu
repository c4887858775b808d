// The consumer of INT8 codes with one scale per row on both sides: an INT8
// product on the 5th-generation tensor cores.
//
//   y[t][c] = RN(RN(RN(sum_k a[t][k] b[c][k]) s_a[t]) s_b[c])
//
// a: token rows, b: channel rows (a weight), both as ss24_quantize_int writes
// them with bits 8 and group 0. The sum is exact in 32-bit integers (128^2 k <
// 2^31); it is rounded once to binary32 and once by each scale, and once more
// where y is bf16.
//
// Roles. The channels are the MMA's M (128 rows a CTA), the tokens its N: a
// small token count costs a narrow MMA, not an idle one, and a thread's
// accumulator row is one channel, so that the 32 lanes of a warp write 32
// consecutive channels of a token (whole sectors, any n and ldy).
//
// Two kernels:
//   pair   256 x 256 tiles by pairs of CTAs, persistent, two accumulators in
//          tensor memory. A CTA brings 128 channel rows and 128 token rows and
//          the pair's MMA uses all four halves: 64 bytes a clock to each SM at
//          the MMA's full rate, where one CTA's own 128 x 256 tile needs 96
//          (and reads 96 of the 128 shared memory gives beside that).
//          16384 x 14336 x 4096: 593 us, 3.2 PFLOP/s, the tensor pipe 98% active,
//          at the clock that the power limit leaves (694 us where that is 1.3 GHz).
//   split  128 channels x 16 ... 128 tokens by one CTA, the k axis split over a
//          cluster of up to 8 CTAs and joined through their shared memory: few
//          tokens, where the weight's bytes bound the call and tiles of all of
//          k would leave most SMs idle. One token, 4096 x 4096: 5.1 us (the weight's
//          bytes take 2.6); 77 tokens, 14336 x 4096: 14.8 us (9.3).
#include "serve.cuh"
#include "tcgen05.cuh"

namespace ss24 {

namespace {

constexpr int kBM = 128; // channels per CTA
constexpr int kBK = 128; // k per stage (bytes)

// s32 accumulator, s8 x s8, both K-major
__host__ __device__ constexpr uint32_t i8_idesc(int m, int n)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ uint8_t *align1024(uint8_t *p)
{
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ void store_y(float *y, uint32_t acc, float sa, float sb)
{
    *y = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(acc)), sa), sb);
}
__device__ __forceinline__ void store_y(__nv_bfloat16 *y, uint32_t acc, float sa, float sb)
{
    *y = __float2bfloat16_rn(__fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(acc)), sa), sb));
}

// ---------------------------------------------------------------------------
// pair: 256 channels x 256 tokens by two CTAs
// ---------------------------------------------------------------------------

constexpr int kPairThreads = 384; // warp 0: loads, warp 1: MMAs, warps 4-11: epilogue
constexpr int kPairN = 256, kPairStages = 6;
constexpr uint32_t kPairStage = 2 * kBM * kBK; // 128 channel rows, 128 token rows
constexpr size_t kPairSmem = 1024 + kPairStages * kPairStage + 512 + 2 * kPairN * 4;
constexpr int kRaster = 8; // token tiles served together

struct PairBars {
    uint64_t full[kPairStages], empty[kPairStages], acc_full[2], acc_empty[2];
};

// Tile i of the persistent order: kRaster token tiles by all channel tiles at a
// time, so that the tiles in flight share rows of both operands in L2.
__device__ __forceinline__ void pair_tile(int64_t i, int64_t tt, int64_t ct, int64_t *t, int64_t *c)
{
    const int64_t band = i / (kRaster * ct), r = i - band * kRaster * ct;
    const int64_t height = tt - band * kRaster < kRaster ? tt - band * kRaster : kRaster;
    *t = band * kRaster + r % height;
    *c = r / height;
}

template <typename Y>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    gemm_int8_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                          const GemmInt8Params p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = align1024(smem_raw);
    PairBars *bars = reinterpret_cast<PairBars *>(stages + kPairStages * kPairStage);
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(bars + 1);
    float *sa = reinterpret_cast<float *>(stages + kPairStages * kPairStage + 512); // [2][kPairN]
    const int tid = threadIdx.x, warp = tc::uniform(tid >> 5), lane = tid & 31;
    const uint32_t rank = tc::cluster_rank();
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int64_t tt = (p.m + kPairN - 1) / kPairN, ct = (p.n + 2 * kBM - 1) / (2 * kBM), tiles = tt * ct;
    const int nk = static_cast<int>((p.k + kBK - 1) / kBK);

    if (tid == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->acc_full[s], 1);
            mbar_init(&bars->acc_empty[s], 16); // the epilogue warps of both CTAs
        }
        fence_barrier_init();
    }
    if (warp == 1)
        tc::alloc_pair(tmem_base, 512);
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = tc::uniform(*tmem_base);
    grid_dependents_launch();
    grid_dependency_wait();
    bool failed = false;

    if (warp == 0 && lane == 0) {
        int it = 0, phase = 0;
        int64_t issued = 0;
        for (int64_t i = pair; i < tiles && !failed; i += pairs) {
            int64_t t, c;
            pair_tile(i, tt, ct, &t, &c);
            const int32_t row_w = static_cast<int32_t>(c * 2 * kBM + rank * kBM);
            const int32_t row_x = static_cast<int32_t>(t * kPairN + rank * kBM);
            for (int kt = 0; kt < nk; ++kt) {
                if (!tc::wait(&bars->empty[it], phase ^ 1, p.wait_limit_ns)) {
                    failed = true;
                    break;
                }
                const uint32_t at = smem_u32(stages + it * kPairStage);
                if (rank == 0)
                    mbar_arrive_expect_tx(&bars->full[it], 2 * kPairStage);
                const uint32_t bar = tc::cluster_addr(smem_u32(&bars->full[it]), 0);
                if (issued != p.test_skip || blockIdx.x != 0)
                    tc::tma_box_pair(at, &map_w, kt * kBK, row_w, bar);
                tc::tma_box_pair(at + kBM * kBK, &map_x, kt * kBK, row_x, bar);
                ++issued;
                if (++it == kPairStages)
                    it = 0, phase ^= 1;
            }
        }
        // the stages' last readers: a CTA leaves only after its copies have landed
        for (int64_t j = issued > kPairStages ? issued - kPairStages : 0; j < issued; ++j)
            if (!tc::wait(&bars->empty[j % kPairStages], (j / kPairStages) & 1, p.wait_limit_ns))
                failed = true;
    } else if (warp == 1 && rank == 0) {
        const bool lead = lane == 0;
        constexpr uint32_t kI = i8_idesc(256, kPairN);
        int it = 0, phase = 0, n = 0;
        for (int64_t i = pair; i < tiles && !failed; i += pairs, ++n) {
            const int a = n & 1;
            if (!tc::wait(&bars->acc_empty[a], ((n >> 1) & 1) ^ 1, p.wait_limit_ns)) {
                failed = true;
                break;
            }
            tc::fence_after();
            for (int kt = 0; kt < nk; ++kt) {
                if (!tc::wait(&bars->full[it], phase, p.wait_limit_ns)) {
                    failed = true;
                    break;
                }
                tc::fence_after();
                const uint32_t at = smem_u32(stages + it * kPairStage);
#pragma unroll
                for (int j = 0; j < kBK / 32; ++j)
                    tc::mma_i8_pair(tmem + a * kPairN, tc::desc_kmajor(at + 32 * j),
                                    tc::desc_kmajor(at + kBM * kBK + 32 * j), kI, (kt | j) != 0, lead);
                tc::commit_pair(&bars->empty[it], lead);
                if (++it == kPairStages)
                    it = 0, phase ^= 1;
            }
            tc::commit_pair(&bars->acc_full[a], lead);
        }
    } else if (warp >= 4) {
        // warps 4-7 take the tile's first 128 tokens, warps 8-11 the others
        const int w = warp & 3, half = (warp - 4) >> 2;
        int n = 0;
        for (int64_t i = pair; i < tiles; i += pairs, ++n) {
            int64_t t, c;
            pair_tile(i, tt, ct, &t, &c);
            const int a = n & 1;
            const int64_t ch = c * 2 * kBM + rank * kBM + 32 * w + lane, t0 = t * kPairN + half * 128;
            const bool on = ch < p.n;
            const float sb = on ? __ldg(p.b_scale + ch) : 0.0f;
            float *const s = sa + a * kPairN + half * 128;
            const int64_t own = t0 + 32 * w + lane;
            s[32 * w + lane] = own < p.m ? __ldg(p.a_scale + own) : 0.0f;
            named_barrier_sync(1 + half, 128);
            // a warp that gave up still meets the others at the barrier above
            failed = failed || !tc::wait_warp(&bars->acc_full[a], (n >> 1) & 1, p.wait_limit_ns);
            if (failed)
                continue;
            tc::fence_after();
            const int64_t room = p.m - t0;
            const int cols = static_cast<int>(room < 0 ? 0 : room < 128 ? room : 128);
            const uint32_t at = tmem + (static_cast<uint32_t>(32 * w) << 16) + a * kPairN + half * 128;
            Y *y = static_cast<Y *>(p.y) + t0 * p.ldy + ch;
#pragma unroll 1
            for (int j0 = 0; j0 < cols; j0 += 32) {
                uint32_t v[32];
                __syncwarp();
                tc::ld32(at + j0, v);
                tc::wait_ld();
                if (j0 + 32 <= cols) {
                    if (on) {
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            store_y(y + q * p.ldy, v[q], s[j0 + q], sb);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 32; ++q)
                        if (on && j0 + q < cols)
                            store_y(y + q * p.ldy, v[q], s[j0 + q], sb);
                }
                y += 32 * p.ldy;
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0)
                tc::arrive_cluster(tc::cluster_addr(smem_u32(&bars->acc_empty[a]), 0));
        }
    }
    if (failed)
        atomicCAS(p.err, 0, kErrGemmWait);
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();
    if (warp == 1) {
        tc::fence_after();
        tc::dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// split: 128 channels x BN tokens, k over the CTAs of a cluster
// ---------------------------------------------------------------------------

constexpr int kSplitThreads = 128;

template <int BN> struct Split {
    static constexpr int kStages = BN <= 64 ? 4 : 6;
    static constexpr int kPerSm = BN <= 64 ? 2 : 1; // CTAs that fit an SM's shared memory
    static constexpr uint32_t kStage = (kBM + BN) * kBK;
    static constexpr uint32_t kCols = BN < 32 ? 32 : BN;
    static constexpr size_t kSmem = 1024 + kStages * kStage + 128 + 4 * BN;
    static_assert(kStages * kStage >= 4 * kBM * (BN < 16 ? 16 : BN), "the stages hold a part's sums");
};

template <int BN, typename Y>
__global__ void __launch_bounds__(kSplitThreads)
    gemm_int8_split_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                           const GemmInt8Params p, const int32_t parts)
{
    using S = Split<BN>;
    constexpr int STAGES = S::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = align1024(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(stages + STAGES * S::kStage);
    uint64_t *empty = full + STAGES;
    uint64_t *accbar = empty + STAGES, *joined = accbar + 1;
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(accbar + 2);
    float *sa = reinterpret_cast<float *>(accbar + 3);

    const int tid = threadIdx.x, warp = tc::uniform(tid >> 5), lane = tid & 31;
    const int rank = static_cast<int>(blockIdx.x % parts);
    const int64_t ct = (p.n + kBM - 1) / kBM, tile = blockIdx.x / parts;
    const int64_t c0 = tile % ct * kBM, t0 = tile / ct * BN;
    const int64_t nk = (p.k + kBK - 1) / kBK;
    const int kt0 = static_cast<int>(nk * rank / parts), kt1 = static_cast<int>(nk * (rank + 1) / parts);

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(accbar, 1);
        mbar_init(joined, 1);
        fence_barrier_init();
    }
    if (warp == 1)
        tc::alloc(tmem_base, S::kCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tc::uniform(*tmem_base);
    grid_dependents_launch();
    grid_dependency_wait();
    bool failed = false;

    if (warp == 0 && lane == 0) {
        int issued = 0;
        for (int kt = kt0; kt < kt1; ++kt, ++issued) {
            const int s = issued % STAGES;
            if (issued >= STAGES && !tc::wait(&empty[s], (issued / STAGES - 1) & 1, p.wait_limit_ns)) {
                failed = true;
                break;
            }
            const uint32_t at = smem_u32(stages + s * S::kStage);
            mbar_arrive_expect_tx(&full[s], S::kStage);
            if (issued != p.test_skip || blockIdx.x != 0)
                tc::tma_box(at, &map_w, kt * kBK, static_cast<int32_t>(c0), &full[s]);
            tc::tma_box(at + kBM * kBK, &map_x, kt * kBK, static_cast<int32_t>(t0), &full[s]);
        }
        // the copies land before the CTA can exit, also where the other warp gave up on one
        for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
            if (!tc::wait(&full[i % STAGES], (i / STAGES) & 1, p.wait_limit_ns))
                failed = true;
    } else if (warp == 1) {
        const bool lead = lane == 0;
        constexpr uint32_t kI = i8_idesc(128, BN);
        for (int i = 0; i < kt1 - kt0; ++i) {
            const int s = i % STAGES;
            if (!tc::wait(&full[s], (i / STAGES) & 1, p.wait_limit_ns)) {
                failed = true;
                break;
            }
            tc::fence_after();
            const uint32_t at = smem_u32(stages + s * S::kStage);
#pragma unroll
            for (int j = 0; j < kBK / 32; ++j)
                tc::mma_i8(tmem, tc::desc_kmajor(at + 32 * j), tc::desc_kmajor(at + kBM * kBK + 32 * j), kI, (i | j) != 0, lead);
            tc::commit(&empty[s], lead);
        }
        tc::commit(accbar, lead);
    }
    __syncwarp();
    const int cols = static_cast<int>(p.m - t0 < BN ? p.m - t0 : BN);
    for (int i = tid; i < cols; i += kSplitThreads)
        sa[i] = p.a_scale[t0 + i];
    const int64_t c = c0 + 32 * warp + lane;
    const bool on = c < p.n;
    const float sb = on ? p.b_scale[c] : 0.0f;
    __syncthreads();
    if (!tc::wait(accbar, 0, p.wait_limit_ns))
        failed = true;
    tc::fence_after();
    const uint32_t acc = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    if (parts == 1) {
#pragma unroll 1
        for (int j0 = 0; j0 < cols; j0 += 16) {
            uint32_t v[16];
            __syncwarp();
            tc::ld16(acc + j0, v);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (on && j0 + i < cols)
                    store_y(static_cast<Y *>(p.y) + (t0 + j0 + i) * p.ldy + c, v[i], sa[j0 + i], sb);
        }
    } else {
        // This part's sums over the stages (all read by now), column j of channel c at
        // 4 (128 j + c). Each CTA answers for a share of the columns; the others' sums of
        // those are added to its own by bulk reductions between the CTAs' shared memories.
        const int share = (cols + parts - 1) / parts;
        const uint32_t sums = smem_u32(stages);
#pragma unroll 1
        for (int j0 = 0; j0 < cols; j0 += 16) {
            uint32_t v[16];
            __syncwarp();
            tc::ld16(acc + j0, v);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) // up to 15 columns of the MMA's behind cols
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(sums + 512 * (j0 + i) + 4 * tid), "r"(v[i]) : "memory");
        }
        const int mine = cols - rank * share < 0 ? 0 : cols - rank * share < share ? cols - rank * share : share;
        if (tid == 0)
            mbar_arrive_expect_tx(joined, static_cast<uint32_t>((parts - 1) * mine * 512));
        tc::fence_proxy();
        __syncthreads();
        tc::cluster_sync();
        if (tid < parts && tid != rank) {
            const int n = cols - tid * share < share ? cols - tid * share : share; // the other's columns
            if (n > 0) {
                const uint32_t from = sums + 512 * share * tid;
                asm volatile("cp.reduce.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes.add.s32"
                             " [%0], [%1], %2, [%3];" ::"r"(tc::cluster_addr(from, tid)),
                             "r"(from), "r"(n * 512), "r"(tc::cluster_addr(smem_u32(joined), tid))
                             : "memory");
            }
        }
        __syncwarp();
        if (!tc::wait(joined, 0, p.wait_limit_ns))
            failed = true;
        for (int j = 0; j < mine; ++j) {
            uint32_t sum;
            const int col = rank * share + j;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sum) : "r"(sums + 512 * col + 4 * tid) : "memory");
            if (on)
                store_y(static_cast<Y *>(p.y) + (t0 + col) * p.ldy + c, sum, sa[col], sb);
        }
        tc::cluster_sync(); // a CTA's sums stay until the reductions have read them
    }
    if (failed)
        atomicCAS(p.err, 0, kErrGemmWait);
    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::dealloc(tmem, S::kCols);
    }
}

template <typename K, typename... A>
cudaError_t launch_gemm(K kern, size_t smem, int64_t grid, int threads, int cluster, cudaStream_t stream, A... args)
{
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kSms = 148;

template <int BN> cudaError_t launch_split(const GemmInt8Params &p, cudaStream_t stream)
{
    CUtensorMap mw, mx;
    if (!tensor_map_bytes(&mw, p.b, p.n, p.k, kBK, kBM) || !tensor_map_bytes(&mx, p.a, p.m, p.k, kBK, BN))
        return cudaErrorInvalidValue;
    const int64_t tiles = ceil_div(p.n, kBM) * ceil_div(p.m, BN), nk = ceil_div(p.k, kBK);
    if (tiles > INT32_MAX / 8)
        return cudaErrorInvalidValue;
    // Parts of k: doubled while all CTAs still run at once and each keeps eight
    // stages of work. One token, 4096 x 4096: 4 parts (of eight stages) 5.1 us, 8
    // parts 5.4, 1 part 9.4; 4096 channels of 14336: 8 parts 12.3, 4 parts 13.7.
    int parts = 1;
    while (parts < 8 && tiles * parts * 2 <= Split<BN>::kPerSm * kSms && nk >= 16 * parts)
        parts *= 2;
    return launch_gemm(p.y_f32 ? gemm_int8_split_kernel<BN, float> : gemm_int8_split_kernel<BN, __nv_bfloat16>,
                       Split<BN>::kSmem, tiles * parts, kSplitThreads, parts, stream, mw, mx, p,
                       static_cast<int32_t>(parts));
}

cudaError_t launch_pair(const GemmInt8Params &p, cudaStream_t stream)
{
    CUtensorMap mw, mx;
    if (!tensor_map_bytes(&mw, p.b, p.n, p.k, kBK, kBM) || !tensor_map_bytes(&mx, p.a, p.m, p.k, kBK, kBM))
        return cudaErrorInvalidValue;
    const int64_t tiles = ceil_div(p.n, 2 * kBM) * ceil_div(p.m, kPairN);
    const int64_t pairs = tiles < kSms / 2 ? tiles : kSms / 2;
    return launch_gemm(p.y_f32 ? gemm_int8_pair_kernel<float> : gemm_int8_pair_kernel<__nv_bfloat16>, kPairSmem, 2 * pairs,
                       kPairThreads, 1, stream, mw, mx, p);
}

} // namespace

cudaError_t launch_gemm_int8(const GemmInt8Params &p, cudaStream_t stream)
{
    // Pairs where their tiles occupy a good part of the SMs. Else the narrowest tile
    // that holds the tokens; above 64 tokens 128 wide ones, which read the weight
    // once, unless they are too few to keep the SMs busy (128 tokens, 1024 channels
    // of 4096: 9.0 us, with 64 wide tiles 7.6; 14336 channels: 15.8 and 17.1).
    if (p.m > 128 && ceil_div(p.n, 2 * kBM) * ceil_div(p.m, kPairN) >= kSms / 4)
        return launch_pair(p, stream);
    if (p.m <= 16)
        return launch_split<16>(p, stream);
    if (p.m <= 32)
        return launch_split<32>(p, stream);
    if (p.m <= 64 || ceil_div(p.n, kBM) * ceil_div(p.m, 128) < 32)
        return launch_split<64>(p, stream);
    return launch_split<128>(p, stream);
}

} // namespace ss24
