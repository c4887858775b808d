// The consumer of INT8 codes with one scale per row on both sides: an INT8
// product on the 5th-generation tensor cores.
//
//   y[t][c] = RN(RN(RN(sum_k a[t][k] b[c][k]) s_a[t]) s_b[c])
//
// a: token rows, b: channel rows (a weight), both as ss24_quantize_int writes
// them with bits 8 and group 0. The sum is exact in 32-bit integers for k <=
// 133,144 (127^2 k < 2^31); it is rounded once to binary32 and once by each
// scale, and once more where y is bf16.
//
// Roles. The channels are the MMA's M (128 rows), the tokens its N: a token
// count that is small costs a narrow MMA, not an idle one, and a thread's
// accumulator row is one channel, so that the 32 lanes of a warp write 32
// consecutive channels of a token (whole sectors, any n and ldy).
#include "serve.cuh"
#include "tcgen05.cuh"

namespace ss24 {

namespace {

constexpr int kBM = 128;      // channels per tile
constexpr int kBK = 128;      // k per stage (bytes)
constexpr int kThreadsG = 128;

template <int BN> struct Shape {
    static constexpr int kStagesG = BN >= 256 ? 4 : 6;
    static constexpr uint32_t kABytes = kBM * kBK, kBBytes = BN * kBK;
    static constexpr uint32_t kStage = kABytes + kBBytes;
    static constexpr uint32_t kTmemCols = BN < 32 ? 32 : BN;
    static constexpr size_t kSmem = kStagesG * kStage + 1024 + 256 + 4 * BN;
};

// s32 accumulator, s8 x s8, both K-major, M = 128, N = BN
template <int BN>
constexpr uint32_t kIdesc = (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(BN >> 3) << 17) |
                            (static_cast<uint32_t>(kBM >> 4) << 24);

template <int BN>
__global__ void __launch_bounds__(kThreadsG, 1)
    gemm_int8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                     const GemmInt8Params p)
{
    using S = Shape<BN>;
    constexpr int STAGES = S::kStagesG;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(stages + STAGES * S::kStage);
    uint64_t *empty = full + STAGES;
    uint64_t *accbar = empty + STAGES;
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(accbar + 1);
    float *sa = reinterpret_cast<float *>(accbar + 4);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kBM, t0 = static_cast<int64_t>(blockIdx.y) * BN;
    const int nk = static_cast<int>((p.k + kBK - 1) / kBK);

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(accbar, 1);
        fence_barrier_init();
    }
    if (warp == 0)
        tc::alloc(tmem_base, S::kTmemCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_base;
    grid_dependency_wait();

    if (warp == 0 && lane == 0) {
        int issued = 0;
        bool failed = false;
        for (int kt = 0; kt < nk; ++kt) {
            const int s = kt % STAGES;
            if (kt >= STAGES && !mbar_wait(&empty[s], ((kt / STAGES) - 1) & 1, p.wait_limit_ns)) {
                failed = true;
                break;
            }
            const uint32_t at = smem_u32(stages + s * S::kStage);
            mbar_arrive_expect_tx(&full[s], S::kStage);
            tc::tma_box(at, &map_w, kt * kBK, static_cast<int32_t>(c0), &full[s]);
            tc::tma_box(at + S::kABytes, &map_x, kt * kBK, static_cast<int32_t>(t0), &full[s]);
            ++issued;
        }
        if (failed) {
            atomicCAS(p.err, 0, kErrGemmWait);
            // the copies already issued land before the CTA can exit
            for (int kt = issued > STAGES ? issued - STAGES : 0; kt < issued; ++kt)
                (void)mbar_wait(&full[kt % STAGES], (kt / STAGES) & 1, p.wait_limit_ns);
        }
    } else if (warp == 1 && lane == 0) {
        for (int kt = 0; kt < nk; ++kt) {
            const int s = kt % STAGES;
            if (!mbar_wait(&full[s], (kt / STAGES) & 1, p.wait_limit_ns)) {
                atomicCAS(p.err, 0, kErrGemmWait);
                break;
            }
            tc::fence_after();
            const uint32_t at = smem_u32(stages + s * S::kStage);
#pragma unroll
            for (int j = 0; j < kBK / 32; ++j)
                tc::mma_i8(tmem, tc::desc_kmajor(at + 32 * j), tc::desc_kmajor(at + S::kABytes + 32 * j), kIdesc<BN>,
                           (kt | j) != 0 ? 1u : 0u);
            tc::commit(&empty[s]);
        }
        tc::commit(accbar);
    }
    __syncwarp();
    for (int i = tid; i < BN; i += kThreadsG)
        sa[i] = t0 + i < p.m ? p.a_scale[t0 + i] : 0.0f;
    __syncthreads();
    if (!mbar_wait(accbar, 0, p.wait_limit_ns) && lane == 0)
        atomicCAS(p.err, 0, kErrGemmWait);
    tc::fence_after();

    const int64_t c = c0 + 32 * warp + lane;
    const float sb = c < p.n ? p.b_scale[c] : 0.0f;
#pragma unroll 1
    for (int j0 = 0; j0 < BN; j0 += 16) {
        if (t0 + j0 >= p.m)
            break;
        uint32_t v[16];
        tc::ld16(tmem + (static_cast<uint32_t>(32 * warp) << 16) + j0, v);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t t = t0 + j0 + i;
            if (t < p.m && c < p.n) {
                const float r = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(v[i])), sa[j0 + i]), sb);
                if (p.y_f32)
                    static_cast<float *>(p.y)[t * p.ldy + c] = r;
                else
                    static_cast<__nv_bfloat16 *>(p.y)[t * p.ldy + c] = __float2bfloat16_rn(r);
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after();
        tc::dealloc(tmem, S::kTmemCols);
    }
}

bool encode_rows(CUtensorMap *map, const int8_t *base, int64_t rows, int64_t k, uint32_t box_rows)
{
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    if (!encode)
        return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
    cuuint64_t stride[1] = {static_cast<cuuint64_t>(k)};
    cuuint32_t box[2] = {kBK, box_rows};
    cuuint32_t one[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(base), dims, stride, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN> cudaError_t launch_bn(const GemmInt8Params &p, cudaStream_t stream)
{
    using S = Shape<BN>;
    CUtensorMap mw, mx;
    if (!encode_rows(&mw, p.b, p.n, p.k, kBM) || !encode_rows(&mx, p.a, p.m, p.k, BN))
        return cudaErrorInvalidValue;
    auto kern = gemm_int8_kernel<BN>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.n + kBM - 1) / kBM), static_cast<unsigned>((p.m + BN - 1) / BN));
    cfg.blockDim = dim3(kThreadsG);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, mw, mx, p);
}

} // namespace

cudaError_t launch_gemm_int8(const GemmInt8Params &p, cudaStream_t stream)
{
    if (p.m <= 16)
        return launch_bn<16>(p, stream);
    if (p.m <= 64)
        return launch_bn<64>(p, stream);
    if (p.m <= 128)
        return launch_bn<128>(p, stream);
    return launch_bn<256>(p, stream);
}

} // namespace ss24
