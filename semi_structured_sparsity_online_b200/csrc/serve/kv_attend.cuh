// What the attention kernels share: decoding of codes, query rows.
#pragma once

#include "serve.cuh"

namespace ss24 {

constexpr float kLn2 = 0.693147180559945f;

// four 8-bit codes -> two fp16 pairs, exact
template <bool FP8> __device__ __forceinline__ void codes4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if constexpr (FP8) {
        lo = e4m3x2h_to_f16x2(static_cast<uint16_t>(w));
        hi = e4m3x2h_to_f16x2(static_cast<uint16_t>(w >> 16));
    } else {
        // 0x6400 | u is 1024 + u; u = code + 128
        const uint32_t u = w ^ 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480)); // 1152
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    }
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Row r of a (sequence, KV head): its token row, its query head, and the keys
// it sees.
struct RowAt {
    int64_t token;
    int32_t head, limit;
};
__device__ __forceinline__ RowAt row_at(const KvAttendParams &p, int64_t r, int h, int32_t first, int32_t count,
                                        int32_t len)
{
    const int32_t i = static_cast<int32_t>(r / p.group);
    RowAt a;
    a.token = first + i;
    a.head = h * p.group + static_cast<int32_t>(r - static_cast<int64_t>(i) * p.group);
    const int32_t seen = len - count + i + 1;
    a.limit = !p.causal ? len : seen < 0 ? 0 : seen;
    return a;
}

// Sequences in order of falling length (equal ones by number), so that the CTAs
// of a long one do not start last: 64 sequences between 1024 and 8192 tokens take
// 98 us instead of 120, with 40 rows each over up to 4000 keys 161 instead of 180.
// One thread counts for one sequence. More sequences even out without, and the count
// takes longer: 300 with 20 new tokens over up to 1000 keys 53 us, in order 73; 256
// with one over up to 300 keys 15 and 22, 200 over up to 4000 keys 99 and 92.
// `room`: shared memory for a number per thread.
constexpr int kMostOrdered = 128; // no more than a CTA's threads
__device__ __forceinline__ int32_t longest_first(const KvBatch &b, uint32_t rank, int32_t *room)
{
    const int n = static_cast<int>(b.seqs), tid = threadIdx.x;
    if (n == 1 || n > kMostOrdered)
        return rank;
    const int32_t mine = tid < n ? __ldg(b.lengths + tid) : -1;
    room[tid] = mine;
    __syncthreads();
    uint32_t before = 0;
    if (tid < n)
        for (int i = 0; i < n; ++i)
            before += room[i] > mine || (room[i] == mine && i < tid);
    __syncthreads();
    if (tid < n && before == rank)
        room[0] = tid;
    __syncthreads();
    const int32_t s = room[0];
    __syncthreads();
    return s;
}

// Attention on the 5th-generation tensor cores, tiles of 128 or 256 rows
// (kv_attend_tiles.cu).
constexpr int kTileRows = 256;
// Whether pairs of CTAs take 512 rows together: heads of 128 and more rows than
// one CTA holds.
inline bool kv_attend_pairs(const KvAttendParams &p)
{
    return p.cache.d == 128 && p.batch.max_new * p.group > kTileRows;
}
cudaError_t launch_kv_attend_tiles(const KvAttendParams &p, cudaStream_t stream);

} // namespace ss24
