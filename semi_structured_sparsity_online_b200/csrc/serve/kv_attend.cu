// Attention of new tokens over the 8-bit paged cache, few query rows per
// (sequence, KV head): one warp works on 16 keys (heads of 64: 32) at a time.
//
//   x[r][j] = scale q_r . (k_j s_k) log2(e),  s_k, s_v: the scales of j's page
//   o_r = sum_j 2^(x[r][j]) (v_j s_v) / sum_j 2^(x[r][j]),  lse_r = ln 2 log2 sum_j 2^(x[r][j])
//
// Rows. The queries of the heads that share a KV head (group) and of several
// new tokens are rows of one tile: row r is token r / group, head r % group.
// Both products run on the tensor cores with the keys (or the head dimension)
// as the MMA's M and 8 rows as its N, so that 4 or 8 rows leave nothing idle.
// Each warp walks over its own 16-key groups through its own ring of TMA boxes
// (swizzled, so that the fragment reads hit distinct banks) and waits for no
// other warp until its end; the MMA's k order is free as long as both operands
// agree, so a fragment is 16 bytes of a key as they lie.
// Codes are exact in fp16 (|code| <= 128, or E4M3). q is held in fp16 after a
// power-of-two scaling of its row by its largest magnitude: what that drops is
// below 2^-24 of that magnitude.
//
// The weights of the second product carry the V scale: w = 2^(x + log2 s_v -
// M), rounded once to fp16, with a reference point M that follows the keys at
// hand (kv_attend.cuh). The denominator sums w / s_v in binary32. Scales s_v
// below 2^-100 count as 2^-100.
//
// Bound by memory where there is enough of it: 64 sequences of 1024 to 8192 keys,
// 8 KV heads of 128, INT8: 96 - 102 us, 5.8 TB/s (0.88 of the measured copy);
// 131072 keys, E4M3: 53 - 55 us, 5.0 TB/s. A 16-key group takes 380 instructions, a
// third of them the conversion of the codes (ALU pipe 51% active).
#include "kv_attend.cuh"
#include "tcgen05.cuh"

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

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

constexpr int kRowWarps = 8;               // they take a part's 16-key groups in turn
constexpr int kRows = 8;                   // of a tile: the MMA's N

template <int D> struct RowShape {
    static constexpr int kRing = 3;
    // Groups of 16 keys a warp takes at a time. Two share the wait, the vote and the
    // maxima: 64 sequences of 8192 keys, E4M3, heads of 64 take 105 us, one by one 116.
    // Heads of 128 have no registers for two.
    static constexpr int kTogether = D == 128 ? 1 : 2;
    static constexpr uint32_t kBox = 16 * D;      // 16 keys of K or of V
    static constexpr uint32_t kGroup = 2 * kBox;
    static constexpr uint32_t kSlot = kTogether * kGroup;
    static constexpr int kPerSm = 2;
    // afterwards the boxes hold the warps' sums [warp][row][D + 4]
    static constexpr uint32_t kSums = kRowWarps * kRows * (D + 4) * 4;
    static constexpr uint32_t kTiles =
        kRowWarps * kRing * kSlot > kSums ? kRowWarps * kRing * kSlot : kSums;
    static constexpr size_t kSmem = 1024 + kTiles + 2 * kRowWarps * kRows * 4 + kRowWarps * kRing * 8;
};

// 16-byte chunk c of row r in a swizzled box.
template <int D> __device__ __forceinline__ uint32_t box_chunk(int r, int c)
{
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kRowWarps * 32, RowShape<D>::kPerSm)
    kv_attend_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                          const KvAttendParams p)
{
    using S = RowShape<D>;
    constexpr int ROWS = kRows, MT = D / 16, WARPS = kRowWarps, RING = S::kRing, U = S::kTogether;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t *gen = smem_raw + (base - smem_u32(smem_raw));
    float(*sm_o)[ROWS][D + 4] = reinterpret_cast<float(*)[ROWS][D + 4]>(gen);
    float(*sm_m)[ROWS] = reinterpret_cast<float(*)[ROWS]>(gen + S::kTiles);
    float(*sm_l)[ROWS] = sm_m + WARPS;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm_l + WARPS) + RING * (threadIdx.x >> 5); // this warp's
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    uint32_t b = blockIdx.x;
    const int split = b % p.splits;
    b /= p.splits;
    const int h = b % p.cache.kv_heads;
    b /= p.cache.kv_heads;
    const int tile = b % p.row_tiles;
    grid_dependents_launch();
    grid_dependency_wait();
    const int64_t s = longest_first(p.batch, b / p.row_tiles, reinterpret_cast<int32_t *>(gen));

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

    // this warp's rounds of U groups: keys kb + 16 U (warp + WARPS r) on; the last
    // round's second group may lie behind ke
    const int all = ke > kb ? static_cast<int>((ke - kb + 16 * U - 1) / (16 * U)) : 0;
    const int rounds = all > warp ? (all - warp + WARPS - 1) / WARPS : 0;
    if (lane == 0) {
        for (int i = 0; i < RING; ++i)
            mbar_init(&full[i], 1);
        fence_barrier_init();
        tc::fence_proxy(); // the copies overwrite longest_first's room
    }
    __syncwarp();
    bool failed = false;
    const int32_t *table = p.batch.table + s * p.batch.table_ld;
    const uint32_t ring = base + warp * (RING * S::kSlot);
    auto key_of = [&](int i) {
        return static_cast<int32_t>(kb) + 16 * (U * (warp + WARPS * (i / U)) + i % U);
    };
    auto there = [&](int i) { return i < U * rounds && key_of(i) < ke; };

    // 32 groups at a time: lane i holds the page and scales of group 32 n + i;
    // the next 32 pages are loaded meanwhile. -1: outside the cache, no keys.
    auto load_id = [&](int i) { return there(i) ? __ldg(table + (key_of(i) >> p.cache.log2_page)) : -1; };
    int32_t id = load_id(lane), id_next = load_id(32 + lane);
    float s_k, s_v, s_inv;
    auto load_scales = [&] {
        const bool on = id >= 0 && id < p.cache.pages;
        const int64_t ph = on ? static_cast<int64_t>(id) * p.cache.kv_heads + h : 0;
        s_k = on ? __ldg(p.cache.scales[0] + ph) : 0.0f;
        const float v = on ? fmaxf(__ldg(p.cache.scales[1] + ph), 0x1p-100f) : 1.0f;
        s_v = log2f(v);
        s_inv = __frcp_rn(v) * kWeightUnit;
        if (!on)
            id = -1;
    };
    // Copies of round r's groups, on pages `page`, into a slot.
    auto fetch = [&](int r, int slot, const int32_t (&page)[U]) {
        if (lane == 0) {
            uint64_t *bar = &full[slot];
            int on = 0;
#pragma unroll
            for (int u = 0; u < U; ++u)
                on += page[u] >= 0;
            if (on == 0) {
                mbar_arrive(bar);
            } else {
                mbar_arrive_expect_tx(bar, on * S::kGroup);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (page[u] >= 0 && (r != p.test_skip || blockIdx.x != 0 || warp != 0)) {
                        const int32_t row = ((page[u] * p.cache.kv_heads + h) << p.cache.log2_page) +
                                            (key_of(U * r + u) & (p.cache.page - 1));
                        const uint32_t at = ring + slot * S::kSlot + u * S::kGroup;
                        tc::tma_box(at, &map_k, 0, row, bar);
                        tc::tma_box(at + S::kBox, &map_v, 0, row, bar);
                    }
            }
        }
    };
    {
        if (there(lane) && (id < 0 || id >= p.cache.pages)) {
            atomicCAS(p.err, 0, kErrPage);
            id = -1;
        }
#pragma unroll
        for (int r = 0; r < RING; ++r) {
            int32_t page[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                page[u] = __shfl_sync(kFull, id, U * r + u);
            if (r < rounds)
                fetch(r, r, page);
        }
    }
    load_scales();

    // q of row g: the 4 values of d that step ks of K's lane layout names
    uint32_t qf[MT][2];
    float fac[2];
    int32_t limit[2];
    {
        float v[MT][4];
        float amax = 0.0f;
        const bool on = g < live;
        const RowAt a = row_at(p, row0 + (on ? g : 0), h, first, count, len);
        const __nv_bfloat16 *src =
            static_cast<const __nv_bfloat16 *>(p.q.x) + a.token * p.q.token_ld + a.head * p.q.head_ld;
#pragma unroll
        for (int ks = 0; ks < MT; ++ks) {
            const uint2 w =
                __ldg(reinterpret_cast<const uint2 *>(src + (D / 4) * q + 4 * ks));
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
        const int e = query_exponent(static_cast<int>(__float_as_uint(amax) >> 23) - 127);
        const float down = exp2_int(-e);
#pragma unroll
        for (int ks = 0; ks < MT; ++ks) {
            qf[ks][0] = pack_f16(v[ks][0] * down, v[ks][1] * down);
            qf[ks][1] = pack_f16(v[ks][2] * down, v[ks][3] * down);
        }
        const float f = p.scale_log2 * exp2_int(e);
        // the accumulators' rows of this lane: 2q, 2q + 1
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            fac[i] = __shfl_sync(kFull, f, (2 * q + i) * 4);
            const int r = 2 * q + i;
            limit[i] = r < live ? row_at(p, row0 + r, h, first, count, len).limit : 0;
        }
    }
    const int32_t low = row_at(p, row0, h, first, count, len).limit; // the least any row sees

    float o[MT][4] = {};
    float m[2] = {-1e30f, -1e30f}, l[2] = {0.0f, 0.0f};
    // the highest m of each row, until the warps' sums are joined
    if (g == 0)
        sm_m[warp][2 * q] = sm_m[warp][2 * q + 1] = -1e30f;
    __syncwarp();

    int slot = 0, phase = 0, r = 0;
    for (; r < rounds; ++r) {
        const int first_group = U * r;
        if (r > 0 && (first_group & 31) == 0) {
            id = id_next;
            if (there(first_group + lane) && (id < 0 || id >= p.cache.pages))
                atomicCAS(p.err, 0, kErrPage);
            load_scales();
            id_next = load_id(first_group + 32 + lane);
        }
        int32_t page[U];
        float ks_u[U], lsv[U], inv[U];
        bool some = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int from = (first_group & 31) + u;
            page[u] = __shfl_sync(kFull, id, from);
            ks_u[u] = __shfl_sync(kFull, s_k, from);
            lsv[u] = __shfl_sync(kFull, s_v, from);
            inv[u] = __shfl_sync(kFull, s_inv, from);
            some |= page[u] >= 0;
        }
        if (!tc::wait_warp(&full[slot], phase, p.wait_limit_ns)) {
            failed = true;
            break;
        }
        const uint32_t at = ring + slot * S::kSlot;
        if (some) {
            float sc[U][4] = {};
            const int32_t key = key_of(first_group);
            bool edge = key + 16 * U > ke || key + 16 * U > low;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // two chains of products, even and odd steps
                float sd[4] = {};
                uint4 wa, wb;
                const uint32_t k_at = at + u * S::kGroup;
                edge |= page[u] < 0;
#pragma unroll
                for (int ks = 0; ks < MT; ++ks) {
                    if ((ks & 3) == 0) {
                        wa = lds16(k_at + box_chunk<D>(g, (D / 64) * q + ks / 4));
                        wb = lds16(k_at + box_chunk<D>(g + 8, (D / 64) * q + ks / 4));
                    }
                    const uint32_t a = (ks & 3) == 0 ? wa.x : (ks & 3) == 1 ? wa.y : (ks & 3) == 2 ? wa.z : wa.w;
                    const uint32_t c = (ks & 3) == 0 ? wb.x : (ks & 3) == 1 ? wb.y : (ks & 3) == 2 ? wb.z : wb.w;
                    uint32_t a0, a1, a2, a3;
                    codes4_to_f16<FP8>(a, a0, a2);
                    codes4_to_f16<FP8>(c, a1, a3);
                    mma_f16((ks & 1) ? sd : sc[u], a0, a1, a2, a3, qf[ks][0], qf[ks][1]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sc[u][i] = fmaf(sc[u][i] + sd[i], ks_u[u] * fac[i & 1], lsv[u]);
            }
            // sc: (key g, rows 2q, 2q + 1), (key g + 8, the same rows)
            if (edge)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t j = key + 16 * u + g + 8 * (i >> 1);
                        if (page[u] < 0 || j >= limit[i & 1] || j >= ke)
                            sc[u][i] = -INFINITY;
                    }
            float most[2]; // of this lane's keys
            bool off = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                most[i] = fmaxf(sc[0][i], sc[0][i + 2]);
#pragma unroll
                for (int u = 1; u < U; ++u)
                    most[i] = fmaxf(most[i], fmaxf(sc[u][i], sc[u][i + 2]));
                off |= weight_off(m[i], most[i]);
            }
            // The rows stay where no lane's keys are too high and a lane of each row has some
            // that are high enough.
            bool move = __any_sync(kFull, off);
            if (move) {
                const bool high = most[0] - m[0] > kWeightMost || most[1] - m[1] > kWeightMost;
                uint32_t near0 = __ballot_sync(kFull, most[0] - m[0] >= kWeightLeast);
                uint32_t near1 = __ballot_sync(kFull, most[1] - m[1] >= kWeightLeast);
                near0 |= near0 >> 16, near1 |= near1 >> 16;
                near0 |= near0 >> 8, near1 |= near1 >> 8;
                near0 |= near0 >> 4, near1 |= near1 >> 4;
                move = __any_sync(kFull, high) || (near0 & near1 & 15) != 15;
            }
            if (move) {
                const bool may_fall = __all_sync(kFull, fmaxf(l[0], l[1]) < kFallBelow);
                float to[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = most[i];
                    x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
                    to[i] = weight_reference(m[i], x, sm_m[warp][2 * q + i], may_fall);
                }
                if (__any_sync(kFull, to[0] != m[0] || to[1] != m[1])) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float f = exp2_approx(m[i] - to[i]);
                        m[i] = to[i];
                        l[i] *= f;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            o[mt][i] *= f;
                            o[mt][i + 2] *= f;
                        }
                        if (g == 0)
                            sm_m[warp][2 * q + i] = fmaxf(sm_m[warp][2 * q + i], to[i]);
                    }
                    __syncwarp();
                }
            }
            uint32_t pf[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = exp2_approx(sc[u][i] - m[i & 1]);
                l[0] = fmaf(w[0] + w[2], inv[u], l[0]);
                l[1] = fmaf(w[1] + w[3], inv[u], l[1]);
                pf[u][0] = transpose8x8(pack_f16(w[0], w[1]));
                pf[u][1] = transpose8x8(pack_f16(w[2], w[3]));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t v_at = at + u * S::kGroup + S::kBox;
                // of V, lane (g, q) takes the D / 8 bytes at g D / 8 of keys 2q, 2q + 1, 2q + 8, 2q + 9
                uint32_t v[4][D / 32];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 2 * q + (i & 1) + 8 * (i >> 1);
                    if constexpr (D == 128) {
                        const uint4 w = lds16(v_at + box_chunk<D>(r, g));
                        v[i][0] = w.x, v[i][1] = w.y, v[i][2] = w.z, v[i][3] = w.w;
                    } else {
                        const uint2 w = lds8(v_at + box_chunk<D>(r, g >> 1) + 8 * (g & 1));
                        v[i][0] = w.x, v[i][1] = w.y;
                    }
                }
                if (page[u] < 0 || (FP8 && key + 16 * u + 16 > ke)) {
                    // slots behind the last token may hold NaN codes, and a group without a page
                    // what its place in the ring held before
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (page[u] < 0 || key + 16 * u + 2 * q + (i & 1) + 8 * (i >> 1) >= ke)
#pragma unroll
                            for (int w = 0; w < D / 32; ++w)
                                v[i][w] = 0;
                }
                // m tile mt: rows g, g + 8 are elements g D / 8 + 2 mt, + 1
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    uint32_t lo[4], hi[4];
                    pairs4_to_f16<FP8>(v[0][w], v[1][w], lo);
                    pairs4_to_f16<FP8>(v[2][w], v[3][w], hi);
                    mma_f16(o[2 * w], lo[0], lo[1], hi[0], hi[1], pf[u][0], pf[u][1]);
                    mma_f16(o[2 * w + 1], lo[2], lo[3], hi[2], hi[3], pf[u][0], pf[u][1]);
                }
            }
        }
        // every lane has read the slot: the round RING on takes it
        const int n = U * (r + RING);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t id_n = __shfl_sync(kFull, (n ^ first_group) & ~31 ? id_next : id, (n & 31) + u);
            page[u] = id_n < p.cache.pages ? id_n : -1;
        }
        if (r + RING < rounds)
            fetch(r + RING, slot, page);
        if (++slot == RING)
            slot = 0, phase ^= 1;
    }
    // a wait that ran out: the copies on their way land before the CTA exits
    if (failed)
        for (int n = r + RING; r < n && r < rounds; ++r) {
            (void)tc::wait(&full[slot], phase, p.wait_limit_ns / 8);
            if (++slot == RING)
                slot = 0, phase ^= 1;
        }
    // every warp is through with the boxes before they take the sums
    __syncthreads();
    // the warps' sums joined
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(kFull, l[i], 4);
        l[i] += __shfl_xor_sync(kFull, l[i], 8);
        l[i] += __shfl_xor_sync(kFull, l[i], 16);
        const int r = 2 * q + i;
        if (g == 0)
            sm_m[warp][r] = m[i], sm_l[warp][r] = l[i];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            *reinterpret_cast<float2 *>(&sm_o[warp][r][g * (D / 8) + 2 * mt]) =
                make_float2(o[mt][i], o[mt][i + 2]);
    }
    if (failed)
        atomicCAS(p.err, 0, kErrAttendWait);
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
        const bool any = den != 0.0f; // NaN from a NaN in q
        const float inv = any ? weight_inverse(den) : 0.0f;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        const float lse2 = any ? top + kWeightUnitLog + log2f(den) : -INFINITY;
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

// Joins the parts of the key axis: one CTA per (token, query head). Weights of
// the parts first, then the warps sum every kJoinWarps-th part each, several
// loads in flight.
constexpr int kJoinWarps = 4, kMaxParts = 1024;

template <int D> __global__ void __launch_bounds__(kJoinWarps * 32) kv_attend_join_kernel(const KvAttendParams p)
{
    __shared__ float weight[kMaxParts];
    __shared__ float part_top[kJoinWarps], part_den[kJoinWarps];
    __shared__ float sums[kJoinWarps][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = kJoinWarps * 32;
    const int32_t heads = p.cache.kv_heads * p.group;
    const int64_t flat = blockIdx.x;
    const int32_t token = blockIdx.x / heads, head = blockIdx.x - token * heads;
    __shared__ int32_t owned;
    if (tid == 0)
        owned = 0;
    grid_dependency_wait();
    __syncthreads();
    // the token's sequence; tokens of none, or of one that breaks a bound, have no parts
    for (int64_t s = tid; s < p.batch.seqs; s += threads) {
        int32_t first, count, len;
        if (token >= __ldg(p.batch.starts + s) && token < __ldg(p.batch.starts + s + 1) &&
            kv_sequence(p.batch, s, p.err, &first, &count, &len))
            owned = 1;
    }
    __syncthreads();
    if (!owned)
        return;
    const float *lse = p.part_lse + flat * p.splits;
    float top = -INFINITY;
    for (int i = tid; i < p.splits; i += threads) {
        const float x = lse[i];
        weight[i] = x;
        top = fmaxf(top, x);
    }
    for (int o = 16; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if (lane == 0)
        part_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w)
        top = fmaxf(top, part_top[w]);
    constexpr int PER = D / 32;
    float acc[PER] = {};
    float den = 0.0f;
    const float *src = p.part_o + flat * p.splits * D + lane * PER;
#pragma unroll 4
    for (int i = warp; i < p.splits; i += kJoinWarps) {
        // a part without keys for the row has weight 0 and finite sums (zeros)
        const float w = weight[i] == -INFINITY ? 0.0f : exp2_approx(weight[i] - top);
        float x[PER];
        if constexpr (PER == 4)
            *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(src + static_cast<int64_t>(i) * D);
        else
            *reinterpret_cast<float2 *>(x) = *reinterpret_cast<const float2 *>(src + static_cast<int64_t>(i) * D);
        den += w;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            acc[j] = fmaf(w, x[j], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
        sums[warp][lane * PER + j] = acc[j];
    if (lane == 0)
        part_den[warp] = den;
    __syncthreads();
    if (tid >= D / 2)
        return;
    float2 r = make_float2(0.0f, 0.0f);
    den = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        r.x += sums[w][2 * tid], r.y += sums[w][2 * tid + 1];
        den += part_den[w];
    }
    const float inv = den != 0.0f ? __frcp_rn(den) : 0.0f;
    __nv_bfloat16 *dst =
        static_cast<__nv_bfloat16 *>(p.out.x) + token * p.out.token_ld + head * p.out.head_ld + 2 * tid;
    *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(r.x * inv, r.y * inv);
    if (p.lse && tid == 0)
        p.lse[flat] = den != 0.0f ? kLn2 * (top + log2f(den)) : -INFINITY;
}

// The same for few parts of many rows, where a CTA per row would be mostly start: a
// warp joins a row, a CTA kFewHeads rows of a token. Lane i has the weight of part i.
// A chunk of 512 tokens over 4000 keys, 32 heads of 128: 54.7 us, with the kernel
// above 65.3; 64 tokens 29.7 and 28.3.
constexpr int kFewParts = 8, kFewHeads = 16;
constexpr int64_t kManyRows = 148 * 16; // more than the CTAs above that run at once

template <int D> __global__ void __launch_bounds__(kJoinWarps * 32) kv_attend_join_few_kernel(const KvAttendParams p)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t heads = p.cache.kv_heads * p.group, ctas = (heads + kFewHeads - 1) / kFewHeads;
    const int32_t token = blockIdx.x / ctas, head0 = (blockIdx.x - token * ctas) * kFewHeads;
    grid_dependency_wait();
    // the token's sequence; tokens of none, or of one that breaks a bound, have no parts
    bool mine = false;
    for (int64_t s = tid; s < p.batch.seqs; s += kJoinWarps * 32) {
        int32_t first, count, len;
        mine |= token >= __ldg(p.batch.starts + s) && token < __ldg(p.batch.starts + s + 1) &&
                kv_sequence(p.batch, s, p.err, &first, &count, &len);
    }
    if (!__syncthreads_or(mine))
        return;
    constexpr int PER = D / 32;
    const int32_t end = head0 + kFewHeads < heads ? head0 + kFewHeads : heads;
#pragma unroll 2
    for (int32_t head = head0 + warp; head < end; head += kJoinWarps) {
        const int64_t flat = static_cast<int64_t>(token) * heads + head;
        const float *src = p.part_o + flat * p.splits * D + lane * PER;
        float x[kFewParts][PER];
#pragma unroll
        for (int i = 0; i < kFewParts; ++i)
            if (i < p.splits) {
                if constexpr (PER == 4)
                    *reinterpret_cast<float4 *>(x[i]) = *reinterpret_cast<const float4 *>(src + i * D);
                else
                    *reinterpret_cast<float2 *>(x[i]) = *reinterpret_cast<const float2 *>(src + i * D);
            }
        const float lse = lane < p.splits ? p.part_lse[flat * p.splits + lane] : -INFINITY;
        float top = lse;
        for (int o = kFewParts / 2; o; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        top = __shfl_sync(kFull, top, 0);
        const float w = lse == -INFINITY ? 0.0f : exp2_approx(lse - top); // 0 for a part without keys
        float den = 0.0f, acc[PER] = {};
#pragma unroll
        for (int i = 0; i < kFewParts; ++i)
            if (i < p.splits) {
                const float wi = __shfl_sync(kFull, w, i);
                den += wi;
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    acc[j] = fmaf(wi, x[i][j], acc[j]);
            }
        const bool any = den != 0.0f;
        const float inv = any ? __frcp_rn(den) : 0.0f;
        __nv_bfloat16 *dst =
            static_cast<__nv_bfloat16 *>(p.out.x) + token * p.out.token_ld + head * p.out.head_ld + lane * PER;
        uint32_t y[PER / 2];
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * j] * inv, acc[2 * j + 1] * inv);
            y[j] = *reinterpret_cast<const uint32_t *>(&b);
        }
        if constexpr (PER == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(y[0], y[1]);
        else
            *reinterpret_cast<uint32_t *>(dst) = y[0];
        if (p.lse && lane == 0)
            p.lse[flat] = any ? kLn2 * (top + log2f(den)) : -INFINITY;
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename K, typename... A>
cudaError_t launch(K kern, int64_t grid, int threads, size_t smem, cudaStream_t stream, A... args)
{
    if (smem > 0) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Up to 32 rows per (sequence, KV head) go to the kernel above, more to the
// tensor-memory kernel, whose time hardly depends on the rows up to 256. 32 rows
// here and 40 there, INT8 heads of 128: 16 sequences of 1024 to 8192 keys 88 and 127
// us, 32 of up to 1000 keys 17 and 22; 16 sequences of 8192 keys 175 and 129, one
// of 30000 47 and 38.
bool wide(const KvAttendParams &p) { return p.batch.max_new * p.group > 32; }

template <int D, bool FP8> cudaError_t launch_rows(const KvAttendParams &p, cudaStream_t stream)
{
    CUtensorMap mk, mv;
    // a cache without pages: maps that no copy uses
    const bool none = p.cache.pages == 0;
    const int64_t rows = none ? 16 : p.cache.pages * p.cache.kv_heads * p.cache.page;
    if (!tensor_map_bytes(&mk, none ? p.q.x : p.cache.codes[0], rows, D, D, 16) ||
        !tensor_map_bytes(&mv, none ? p.q.x : p.cache.codes[1], rows, D, D, 16))
        return cudaErrorInvalidValue;
    return launch(kv_attend_rows_kernel<D, FP8>, p.batch.seqs * p.cache.kv_heads * p.row_tiles * p.splits,
                  kRowWarps * 32, RowShape<D>::kSmem, stream, mk, mv, p);
}

} // namespace

void kv_attend_plan(KvAttendParams *p)
{
    const int64_t rows = p->batch.max_new * p->group;
    const int64_t len = p->batch.max_len > 0 ? p->batch.max_len : 1;
    const int pair = wide(*p) && kv_attend_pairs(*p) ? 2 : 1;
    const int64_t tile = wide(*p) ? pair * kTileRows : kRows;
    p->row_tiles = static_cast<int32_t>(ceil_div(rows, tile));
    const int64_t ctas = p->batch.seqs * p->cache.kv_heads * p->row_tiles;
    // Parts of the key axis: as many CTAs as run at once and no more, of 512 keys
    // or more. A second wave costs its start and end (131072 keys, 8 heads, 8 rows
    // each: 53 us in one wave of 296, 58 in two, 68 in four). Smaller parts save
    // little on the device and cost the join's launch (500 keys: 7.4 us in one
    // part, 7.8 in two; 1000 keys: 9.4 in two, 8.2 in four).
    // Where that leaves parts of more than 4096 keys, sequences of unequal lengths
    // hold up the wave: two waves of shorter parts (16 sequences of 1024 to 8192
    // keys, 8 heads, 16 rows each: 54 us instead of 86; all of 8192 keys: 99
    // instead of 91). A single sequence stays with one.
    const int64_t step = 128, slots = 148 * (wide(*p) ? 1 : RowShape<128>::kPerSm);
    int64_t splits = ctas > 0 ? slots / (pair * ctas) : 1;
    if (!wide(*p) && ctas > 0 && p->batch.seqs > 1 && (splits == 0 || len / splits > 4096))
        splits = 2 * slots / ctas;
    const int64_t most = ceil_div(len, 4 * step);
    splits = splits > most ? most : splits;
    splits = splits < 1 ? 1 : splits > kMaxParts ? kMaxParts : splits;
    p->split_keys = static_cast<int32_t>(ceil_div(ceil_div(len, splits), step) * step);
    p->splits = static_cast<int32_t>(ceil_div(len, p->split_keys));
}

cudaError_t launch_kv_attend(const KvAttendParams &p, cudaStream_t stream)
{
    cudaError_t e;
    if (wide(p))
        e = launch_kv_attend_tiles(p, stream);
    else if (p.cache.d == 128)
        e = p.cache.fp8 ? launch_rows<128, true>(p, stream) : launch_rows<128, false>(p, stream);
    else
        e = p.cache.fp8 ? launch_rows<64, true>(p, stream) : launch_rows<64, false>(p, stream);
    if (e != cudaSuccess || p.splits <= 1)
        return e;
    const int64_t heads = p.cache.kv_heads * p.group;
    if (p.splits <= kFewParts && p.batch.tokens * heads > kManyRows) {
        const int64_t grid = p.batch.tokens * ceil_div(heads, kFewHeads);
        return p.cache.d == 128 ? launch(kv_attend_join_few_kernel<128>, grid, kJoinWarps * 32, 0, stream, p)
                                : launch(kv_attend_join_few_kernel<64>, grid, kJoinWarps * 32, 0, stream, p);
    }
    const int64_t grid = p.batch.tokens * heads;
    return p.cache.d == 128 ? launch(kv_attend_join_kernel<128>, grid, kJoinWarps * 32, 0, stream, p)
                            : launch(kv_attend_join_kernel<64>, grid, kJoinWarps * 32, 0, stream, p);
}

} // namespace ss24
