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

// The weights of the second product are 2^(y - M) in fp16, y = x + log2 s_v the exponent
// that carries the V scale, M a reference point of the row. fp16 rounds by 2^-11 relative
// from 2^-14 on and by 2^-25 below, and the key with the largest weight may add nothing to
// an element (its code is 0 there), so that the smaller ones have to keep their bits: with
// one M for all keys of a row, at the largest y, a row with 99.9% of its weight on a key of
// zero codes was 8% off over 8192 keys. So M follows the largest y of the keys taken
// together, up and down: it stays where that y is from M - 9 to M + 15. A weight is off by
// no more than 2^-11 of itself or 2^-16 of the largest among those keys (2^-30 where none
// before was larger).
// A move costs the accumulators a pass, so M leaves room for what comes: 10 bits above a y
// that rose, 9 bits below one that fell. A prompt of 8192 tokens, 32 heads of 128, logits
// of deviation 1.2, 3.5 and 9: 555, 604 and 890 us (with M only rising, 8 bits at a time,
// 560, 590 and 691; 5 bits above and 19 below one that rose: 551, 710 and 899).
// M stays within 2^40 of the highest it was, and where the sum of weights over the V scales
// has reached 2^80 (scales below 2^-40) it does not fall: after a fall by 40 it is at most
// 2^120, what follows adds 2^15 2^-7 2^100 a key, so that 2^17 keys stay in binary32's
// range. Weights are lost below 2^-65 of the largest.
constexpr float kWeightMost = 15.0f, kWeightLeast = -9.0f; // y - M that M stays at
constexpr float kWeightRisen = 5.0f, kWeightFallen = 0.0f; // y - M after a move
constexpr float kWeightFall = 40.0f;
constexpr float kFallBelow = 0x1p80f; // the sum of weights that M may still fall with
// The sum of weights over the V scales is taken in units of 2^kWeightUnitLog.
constexpr float kWeightUnitLog = 7.0f, kWeightUnit = 0x1p-7f;
// Whether M may have to move for an exponent y (true for -infinity, too).
__device__ __forceinline__ bool weight_off(float m, float y)
{
    constexpr float kMid = (kWeightMost + kWeightLeast) / 2, kHalf = (kWeightMost - kWeightLeast) / 2;
    return fabsf(y - m - kMid) > kHalf;
}
// M for keys whose largest exponent is y (-infinity: none); `top`: the highest M yet.
// Differences are compared: m + 15 would round where m is large.
__device__ __forceinline__ float weight_reference(float m, float y, float top, bool may_fall)
{
    if (y - m > kWeightMost)
        return y - kWeightRisen;
    return y - m < kWeightLeast && y > -INFINITY && may_fall ? fmaxf(y - kWeightFallen, top - kWeightFall) : m;
}
// What the sum of weighted codes is multiplied with; `sum` in units of 2^kWeightUnitLog.
__device__ __forceinline__ float weight_inverse(float sum)
{
    return sum > 1.0f ? __frcp_rn(sum) * kWeightUnit : __frcp_rn(sum * 0x1p7f);
}

// The power of two by which a row of q is brought into fp16, from the exponent of its
// largest magnitude. At most 112, so that 2^112 times the softmax scale stays finite: bf16's
// largest value is then 65280 in fp16. At least -120, for the same product's sake.
__device__ __forceinline__ int query_exponent(int e) { return e < -120 ? -120 : e > 112 ? 112 : e; }

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
