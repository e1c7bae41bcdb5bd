// k_paged_attn.cu -- softmax attention over listed positions of a paged cache.
//
// For query head h with KV head g: z_t = scale <q_h, sK_t k_t>, o_h = sum_t
// exp(z_t - lse) sV_t v_t, lse = ln sum_t exp(z_t) over the row's listed
// positions t, whose rows the page table locates (sK, sV: the scales of 8-bit
// pages, 1 for bf16).
//
// A unit is (query row, KV head, up to 8 of its query heads); a cluster of C
// CTAs works on it, every warp of the cluster on tiles of 32 keys of its own,
// and no warp waits for another until the end.  Keys are the M side of both
// products and the query heads the N side of 8, so that a group of 8 heads
// fills the warp MMA: S[key][head] = K Q^T, O^T[dim][head] += V^T P.
//   * A lane looks up one key of a tile.  Positions, page table entries, scales
//     and rows all come by asynchronous copies into the warp's own rings in
//     shared memory, each asked for a tile (rows: a stage of 16 keys) before it
//     is used, so that nothing in the loop waits for a load by name: with loads
//     to registers in their place the warps spent over a third of their time at
//     them.  Rings three deep are no faster.
//   * A lane takes 16 consecutive bytes of a K row as fragment elements, which
//     only renames the contraction index (Q's fragments are renamed alike), and
//     of V rows, which renames the output rows; V's pairs along the keys are
//     byte permutations of two rows.  Chunks are XORed with the row so that
//     neither read meets a bank twice.
//   * 8-bit codes become f16, which holds them exactly (the warp MMA's 8-bit
//     form is slower here: 1,024 queries of a 1M context 455 us against 380); a
//     unit's query rows are scaled by a power of two so that f16 holds them too
//     (what falls below f16's subnormals is 2^-37 of their largest element).  sK
//     multiplies the logit in fp32; sV joins the exponent of the weight, w_t =
//     2^(z_t + log2 sV_t - m2), so that the f16 weight of the largest
//     contribution is from 2^7 to 2^15 whatever the scales: a weight is off by
//     2^-11 of itself or, below f16's normal range, by 2^-32 of the largest.  (An
//     eighth of the output's own rounding to bf16 at most: the mean error against
//     64 bits is 1.0006 times that of fp32 weights.  A second f16 for the rest costs
//     3 to 10 %: 8 rows 14.1 us against 14.9, 1,024 rows 370 against 403.)  The
//     denominator sums 2^(z_t - m1) in fp32 with a reference of its own.
//   * bf16 pages: the weight as the sum of two bf16 (2^-17 relative), since one
//     would add as much error as the output's rounding.
//   * The references m1, m2 move only when a value passes them by 2^15: one vote
//     per stage instead of a maximum over lanes.
//   * The logits of a stage are computed beside the products of the stage before
//     (a stage of the ring holds V of 16 keys and K of the next 16), so that two
//     independent chains of MMAs share the warp.
// Warps merge their (m1, m2, sum, O^T) in shared memory; the CTAs of a cluster
// then send each other the slice that the other finishes (distributed shared
// memory, one barrier).
//
// A row is empty when no warp met a key with a slot (PT_EMPTY), whatever its sum; z
// times 0 joins the sum so that infinities and NaN of Q or K are not lost with a weight
// of 0.  All of that is under 1 % of a call.
//
// Bound and measured (B200, 32/4 heads of 128 unless said): 8 rows of 4,612 keys,
// 8-bit, 13.6 us, of which 3.6 before the first product (positions, pages, rows:
// three dependent reads) and 3 in the merge; 32 rows 33 us (4.6 TB/s); 64 rows of
// 16/2 heads in bf16 pages 52 us (5.8 TB/s, 0.89 of a copy's rate: HBM); 251 rows
// of 16/2 heads over 128k in bf16 pages 109 to 117 us by the card (10.1 to 10.9 TB/s of
// rows, most of them from L2); 1,024 rows of 2,564 keys over 1M, 8-bit, 388 to 417 us (6.5
// to 7.0 TB/s of rows: HBM, for rows that list the same bucket seldom run together).  With all warps busy a
// 16-key stage of 8-bit rows issues about 285 instructions, 135 of them on the ALU
// pipe (64 conversions), at 55 to 60 % of the issue slots; CTAs of 8 warps, stages
// of 32 keys and L2 prefetches of later tiles were no faster.
#include <atomic>
#include <type_traits>

#include "paged.cuh"
#include "ptx.cuh"

namespace lsa {

constexpr int PT_WARPS = 4;
constexpr int PT_THREADS = 32 * PT_WARPS;
constexpr int PT_H = 8;             // query heads of a unit
constexpr int PT_MAX_C = 16;        // CTAs of a cluster at most
constexpr float PT_NONE = -3e38f;   // reference before any key's logit
constexpr float PT_EMPTY = -3.4e38f;   // the reference that a warp without a key hands on
constexpr float PT_SLACK = 15.f;    // log2 that a value may pass the reference by
constexpr float PT_UP = 7.f;        // log2 of the f16 weight at its reference's maximum

template <bool E4M3, int D>
struct PagedCfg {
    static constexpr int ROWB = D * (E4M3 ? 1 : 2);   // bytes of one head's row
    static constexpr int KW = ROWB / 16;              // words of a K row per lane
    static constexpr int VW = ROWB / 32;              // words of a V row per lane
    static constexpr int KS = D / 16;                 // contraction steps of S
    static constexpr int DT = D / 16;                 // row tiles of O^T
    static constexpr int LPR = ROWB / 16;             // lanes (16-byte chunks) per row
    static constexpr int RPI = 32 / LPR;              // rows per warp copy
    static constexpr int RI = 16 / RPI;               // copies of 16 rows
    static constexpr int MINB = ROWB > 128 ? 3 : 4;   // CTAs per SM
    static constexpr int HALF = 16 * ROWB;            // bytes of a stage's K (or V)
    static constexpr int STAGE = 2 * HALF;
    static constexpr int RING = 2 * STAGE;            // bytes of a warp's ring
    static constexpr int EPT = PT_H * D / PT_THREADS; // merged elements per thread
    // a warp's positions [2][32], pages [32] and scales [2][2][32] of tiles
    static constexpr int META = 4 * 32 * (E4M3 ? 2 + 1 + 4 : 2 + 1);
    // the slices a CTA of a cluster receives (c slices of ceil(threads / c) threads'
    // elements) and the CTAs' references and sums
    static constexpr int RECV = 4 * EPT * (PT_THREADS + PT_MAX_C), RECV_ML = 4 * 3 * PT_H * PT_MAX_C;
    static constexpr int BYTES =
        PT_WARPS * (RING + META) + RECV + RECV_ML + 4 * 3 * PT_WARPS * PT_H;
    static_assert(4 * PT_H * D <= RING, "a warp's O^T takes its ring's place");
};

struct PagedAttnArgs {
    const __nv_bfloat16* Q;
    int64_t Nq;
    int Hq, hpg, chunks;             // query heads, per KV head, units per KV head
    const int32_t* indices;
    const int32_t* counts;
    int s_max;
    int page_shift;
    float scale_log2;                // scale * log2(e)
    int64_t unit0;                   // this launch's first unit
    __nv_bfloat16* O;
    float* lse;
};

// 4 bytes to shared memory.
__device__ __forceinline__ void copy4(void* dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_addr(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// (not volatile: the compiler orders independent products)
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes to shared memory; zeros for a negative slot (its source is not read).
template <bool FULL>
__device__ __forceinline__ void copy16(uint32_t dst, const char* base, int32_t slot, uint32_t tok_bytes)
{
    if (FULL)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
                     "l"(base + (uint64_t)(uint32_t)slot * tok_bytes)
                     : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %2, 0;\n\t"
            "cp.async.cg.shared.global [%0], [%1], 16, p;\n\t}" ::"r"(dst),
            "l"(base + (uint64_t)(uint32_t)max(slot, 0) * tok_bytes), "r"(slot)
            : "memory");
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t lo_f16x2(uint32_t w) { return e4m3x2_f16x2((uint16_t)w); }
__device__ __forceinline__ uint32_t hi_f16x2(uint32_t w) { return e4m3x2_f16x2((uint16_t)(w >> 16)); }

__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void st_cluster(uint32_t a, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster4(uint32_t a, const float* v)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3])
                 : "memory");
}

template <bool E4M3, int D>
__global__ void __launch_bounds__(PT_THREADS, (PagedCfg<E4M3, D>::MINB))
paged_attn_kernel(lsa_paged_kv kv, PagedAttnArgs a)
{
    using C = PagedCfg<E4M3, D>;
    extern __shared__ __align__(128) char smem[];
    char* tail = smem + PT_WARPS * (C::RING + C::META);
    float* recv = reinterpret_cast<float*>(tail);
    float* recv_ml = reinterpret_cast<float*>(tail + C::RECV);              // [CTA][m1, m2, l][head]
    float* ml_s = reinterpret_cast<float*>(tail + C::RECV + C::RECV_ML);    // [warp] likewise
    uint32_t rank, n_cta;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n_cta));
    grid_dependency();
    // the CTAs of the cluster have started before any is written to
    if (n_cta > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r8 = lane >> 2, t4 = lane & 3;
    const int64_t unit = a.unit0 + blockIdx.x / n_cta;
    const int upr = kv.Hkv * a.chunks;                 // units per row
    const int64_t row = unit / upr;
    const int g = (int)(unit % upr) / a.chunks;
    const int h0 = (int)(unit % upr) % a.chunks * PT_H;
    const int nh = min(PT_H, a.hpg - h0);
    const int64_t hbase = row * a.Hq + (int64_t)g * a.hpg + h0;
    const int64_t b = row / a.Nq;
    const int n = min(max(a.counts[row], 0), a.s_max);
    const int32_t* idx = a.indices + row * a.s_max;
    const int32_t* table = kv.page_table + b * kv.max_pages;
    const uint32_t t_end = (uint32_t)(kv.max_pages << a.page_shift);
    const uint32_t tok_bytes = (uint32_t)kv.Hkv * C::ROWB;
    const char* Kb = (const char*)kv.K + (int64_t)g * C::ROWB;
    const char* Vb = (const char*)kv.V + (int64_t)g * C::ROWB;
    const int n_tiles = (n + 31) / 32;
    const int step = (int)n_cta * PT_WARPS;
    int tile = (int)rank * PT_WARPS + warp;

    // position of this lane's key of tile ti, its page table entry; both clamped
    // into their arrays and checked with the slot (-1: none)
    auto position = [&](int ti) { return idx + min(ti * 32 + lane, a.s_max - 1); };
    auto page = [&](int32_t t) {
        return table + min((uint32_t)t >> a.page_shift, (uint32_t)kv.max_pages - 1u);
    };
    auto slot_of = [&](int32_t t, int32_t pg, int ti) {
        if (ti * 32 + lane >= n) return -1;
        if ((uint32_t)t >= t_end || (uint32_t)pg >= (uint32_t)kv.n_pages) {
            dev_error(kv.status, DEV_BAD_PAGE, (uint32_t)t);
            return -1;
        }
        return (pg << a.page_shift) + (t & (kv.page - 1));
    };
    char* meta = smem + PT_WARPS * C::RING + warp * C::META;
    int32_t* pos_s = reinterpret_cast<int32_t*>(meta) + lane;          // [2][32]
    int32_t* page_s = pos_s + 2 * 32;                                  // [32]
    float* scale_s = reinterpret_cast<float*>(meta) + 3 * 32;          // [2][keys', values'][32]
    // (of slot 0 for a key without a slot, whose logit is replaced)
    auto copy_scales = [&](int at, int32_t slot) {
        if (E4M3) {
            const float* s = kv.scales + (uint64_t)((uint32_t)max(slot, 0) / SCALE_BLOCK) *
                                             (uint32_t)(2 * kv.Hkv) + g;
            copy4(scale_s + at * 64 + lane, s);
            copy4(scale_s + at * 64 + 32 + lane, s + kv.Hkv);
        }
    };
    // A stage of the ring: V of 16 keys, K of the 16 after them; keys without a
    // slot become zeros.  The slots of the rows whose K was copied last serve V's
    // copy of the next stage.
    char* ring = smem + warp * C::RING;
    const int crow = lane / C::LPR, cchunk = lane % C::LPR;
    const uint32_t c_at = crow * C::ROWB + cchunk * 16;
    const uint32_t kc_at = ptx::smem_addr(ring) + (c_at ^ (C::ROWB >= 128 ? (crow & 1) << 6 : 0));
    const uint32_t vc_at = ptx::smem_addr(ring) + C::HALF + (c_at ^ ((crow & 6) << 4));
    const char* Kc = Kb + cchunk * 16;
    const char* Vc = Vb + cchunk * 16;
    int32_t rs[C::RI];
    auto copy_v = [&](int stage, auto full) {
#pragma unroll
        for (int i = 0; i < C::RI; ++i)
            copy16<decltype(full)::value>((vc_at ^ ((i * C::RPI & 6) << 4)) + stage * C::STAGE +
                                              i * C::RPI * C::ROWB,
                                          Vc, rs[i], tok_bytes);
    };
    auto copy_k = [&](int stage, int32_t slot, int half, auto full) {
#pragma unroll
        for (int i = 0; i < C::RI; ++i) {
            rs[i] = __shfl_sync(0xffffffffu, slot, half * 16 + i * C::RPI + crow);
            copy16<decltype(full)::value>(kc_at + stage * C::STAGE + i * C::RPI * C::ROWB, Kc, rs[i],
                                          tok_bytes);
        }
    };
    const std::false_type some{};                      // rows that may have no slot
    const std::true_type full{};

    // Q rows, element order as K's lanes take their bytes: head r8
    uint2 qw[C::KS];
#pragma unroll
    for (int s = 0; s < C::KS; ++s) {
        const int c = E4M3 ? (s / 4) * 64 + t4 * 16 + (s % 4) * 4 : (s / 2) * 32 + t4 * 8 + (s % 2) * 4;
        qw[s] = make_uint2(0u, 0u);
        if (r8 < nh) qw[s] = *reinterpret_cast<const uint2*>(a.Q + (hbase + r8) * D + c);
    }

    // the first tile: in the loop, slot and slot1 are the tile's and the next
    // one's, whose positions and pages have been; the position after them is
    // asked for
    int32_t slot = -1, slot1 = -1;
    if (tile < n_tiles) {
        const int32_t p0 = *position(tile), p1 = *position(tile + step);
        copy4(pos_s, position(tile + 2 * step));
        const int32_t g0 = *page(p0), g1 = *page(p1);
        slot = slot_of(p0, g0, tile);
        copy_scales(0, slot);
        copy_k(1, slot, 0, some);
        ptx::cp_async_commit();
        copy_v(0, some);
        copy_k(0, slot, 1, some);
        ptx::cp_async_commit();
        slot1 = slot_of(p1, g1, tile + step);
    }

    uint32_t qb[C::KS][2];                              // Q fragments
    float factor = a.scale_log2;                        // logit in log2 units of a product
    if (E4M3) {
        float amax = 0.f;                               // of the unit's rows
#pragma unroll
        for (int s = 0; s < C::KS; ++s) {
            amax = fmaxf(amax, finite_abs(__uint_as_float(qw[s].x << 16)));
            amax = fmaxf(amax, finite_abs(__uint_as_float(qw[s].x & 0xffff0000u)));
            amax = fmaxf(amax, finite_abs(__uint_as_float(qw[s].y << 16)));
            amax = fmaxf(amax, finite_abs(__uint_as_float(qw[s].y & 0xffff0000u)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // amax * 2^(13 - e) in [2^13, 2^14)
        const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100);
        const float up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
        factor *= __uint_as_float((uint32_t)(e - 13 + 127) << 23);
#pragma unroll
        for (int s = 0; s < C::KS; ++s) {
            qb[s][0] = pack_f16(__uint_as_float(qw[s].x << 16) * up,
                                __uint_as_float(qw[s].x & 0xffff0000u) * up);
            qb[s][1] = pack_f16(__uint_as_float(qw[s].y << 16) * up,
                                __uint_as_float(qw[s].y & 0xffff0000u) * up);
        }
    } else {
#pragma unroll
        for (int s = 0; s < C::KS; ++s) {
            qb[s][0] = qw[s].x;
            qb[s][1] = qw[s].y;
        }
    }

    float acc[C::DT][4];
#pragma unroll
    for (int j = 0; j < C::DT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    float m1[2] = {PT_NONE, PT_NONE}, m2[2] = {PT_NONE, PT_NONE}, l[2] = {0.f, 0.f};
    bool met = false;                                   // a key with a slot
    // this lane's offsets inside a stage: K rows r8, r8 + 8; V rows 2 t4 ...
    const int k_at = (r8 * C::ROWB + t4 * 16) ^ (C::ROWB >= 128 ? (r8 & 1) << 6 : 0);
    const int v_at = C::HALF + ((2 * t4 * C::ROWB + r8 * (E4M3 ? D / 8 : 16)) ^ (t4 << 5));
    float z[4];                                         // products of keys r8, r8 + 8 with
                                                        // heads 2 t4, 2 t4 + 1
    auto products = [&](const char* st) {
        float y[4] = {0.f, 0.f, 0.f, 0.f};             // a second chain
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = 0.f;
#pragma unroll
        for (int j = 0; j < C::KW / 4; ++j) {
            // chunk 4 j + t4: bit 6 of the offset is j's lowest bit, XORed
            const char* p = st + ((k_at + (j >> 1) * 128) ^ ((j & 1) << 6));
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            const uint4 v = *reinterpret_cast<const uint4*>(p + 8 * C::ROWB);
            const uint32_t k0[4] = {u.x, u.y, u.z, u.w}, k1[4] = {v.x, v.y, v.z, v.w};
            if (E4M3) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_f16(i & 1 ? y : z, lo_f16x2(k0[i]), lo_f16x2(k1[i]), hi_f16x2(k0[i]),
                            hi_f16x2(k1[i]), qb[4 * j + i][0], qb[4 * j + i][1]);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    mma_bf16(i ? y : z, k0[2 * i], k1[2 * i], k0[2 * i + 1], k1[2 * i + 1],
                             qb[2 * j + i][0], qb[2 * j + i][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] += y[i];
    };
    if (tile < n_tiles) {
        ptx::cp_async_wait<1>();
        __syncwarp();
        products(ring + C::STAGE);
    }

    for (int it = 0; tile < n_tiles; tile += step, ++it) {
        const uint32_t valid = __ballot_sync(0xffffffffu, slot >= 0);
        met |= valid != 0u;
        // every row that this tile copies has a slot
        const bool whole = __all_sync(0xffffffffu, slot1 >= 0) && valid == 0xffffffffu;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (half == 1 && tile * 32 + 16 >= n) break;
            __syncwarp();
            {   // the stage read last takes the next one: V of the 16 keys after
                // these, K of the 16 after those
                if (half == 0) {
                    copy4(pos_s + ((it + 1) & 1) * 32, position(tile + 3 * step));
                    copy4(page_s, page(pos_s[(it & 1) * 32]));       // two tiles on
                    copy_scales((it + 1) & 1, slot1);
                }
                if (whole) {
                    copy_v(1 - half, full);
                    copy_k(1 - half, slot1, half, full);
                } else {
                    copy_v(1 - half, some);
                    copy_k(1 - half, slot1, half, some);
                }
                ptx::cp_async_commit();
            }
            // ---- logits, less their references ----
            float d1[4], d2[4], ev[2] = {0.f, 0.f}, kf[2] = {factor, factor};
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (E4M3) {
                    const float* s = scale_s + (it & 1) * 64 + half * 16 + u * 8 + r8;
                    kf[u] *= s[0];
                    ev[u] = __log2f(fmaxf(s[32], 1.17549435e-38f));   // (the least normal)
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d1[i] = fmaf(z[i], kf[i >> 1], -m1[i & 1]);
                d2[i] = E4M3 ? fmaf(z[i], kf[i >> 1], ev[i >> 1] - m2[i & 1]) : d1[i];
            }
            if (valid != 0xffffffffu) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!(valid >> (half * 16 + (i >> 1) * 8 + r8) & 1)) {
                        d1[i] = d2[i] = -INFINITY;
                        z[i] = 0.f;                     // (NaN where Q is not finite)
                    }
            }
            // a key's product of -inf has the weight 0 of no key: infinities and NaN of Q
            // or K reach the sum by themselves
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i & 1] = fmaf(z[i], 0.f, l[i & 1]);
            float top = fmaxf(fmaxf(d1[0], d1[1]), fmaxf(d1[2], d1[3]));
            if (E4M3) top = fmaxf(top, fmaxf(fmaxf(d2[0], d2[1]), fmaxf(d2[2], d2[3])));
            if (__any_sync(0xffffffffu, top > PT_SLACK)) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float n1 = m1[c], n2 = m2[c];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (d1[2 * u + c] > -INFINITY) {
                            const float x = z[2 * u + c] * kf[u];
                            n1 = fmaxf(n1, x);
                            n2 = fmaxf(n2, x + ev[u] - (E4M3 ? PT_UP : 0.f));
                        }
#pragma unroll
                    for (int o = 4; o <= 16; o <<= 1) {
                        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
                        if (E4M3) n2 = fmaxf(n2, __shfl_xor_sync(0xffffffffu, n2, o));
                    }
                    if (!E4M3) n2 = n1;
                    const float f2 = ex2(m2[c] - n2);
                    l[c] *= ex2(m1[c] - n1);
                    m1[c] = n1;
                    m2[c] = n2;
#pragma unroll
                    for (int j = 0; j < C::DT; ++j) {
                        acc[j][c] *= f2;
                        acc[j][c + 2] *= f2;
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int i = 2 * u + c;
                        const bool none = d1[i] == -INFINITY;
                        d1[i] = none ? -INFINITY : fmaf(z[i], kf[u], -n1);
                        d2[i] = none ? -INFINITY : fmaf(z[i], kf[u], ev[u] - n2);
                    }
                }
            }
            // ---- weights, transposed to (keys 2 t4, 2 t4 + 1; head r8) ----
            uint32_t pb[2], pl[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float p0 = ex2(d1[2 * u]), p1 = ex2(d1[2 * u + 1]);
                l[0] += p0;
                l[1] += p1;
                if (E4M3) {
                    pb[u] = ptx::movmatrix_t(pack_f16(ex2(d2[2 * u]), ex2(d2[2 * u + 1])));
                } else {
                    const uint32_t hi = ptx::pack_bf16(p0, p1);
                    pb[u] = ptx::movmatrix_t(hi);
                    pl[u] = ptx::movmatrix_t(ptx::pack_bf16(p0 - __uint_as_float(hi << 16),
                                                            p1 - __uint_as_float(hi & 0xffff0000u)));
                }
            }
            ptx::cp_async_wait<1>();
            __syncwarp();
            const char* st = ring + half * C::STAGE;
            products(st);                               // of the next 16 keys
            // ---- O^T += V^T P: keys 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9 ----
            uint32_t vw[4][C::VW];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                // row 2 t4 + (u & 1) + 8 (u >> 1): the XOR is the lane's
                const char* p = C::ROWB >= 128
                                    ? st + v_at + ((u & 1) + 8 * (u >> 1)) * C::ROWB
                                    : st + ((v_at + 8 * (u >> 1) * C::ROWB) ^ ((u & 1) * C::ROWB));
                if (C::VW == 2) {
                    const uint2 x = *reinterpret_cast<const uint2*>(p);
                    vw[u][0] = x.x;
                    vw[u][1] = x.y;
                } else {
#pragma unroll
                    for (int j = 0; j < C::VW / 4; ++j) {
                        const uint4 x = *reinterpret_cast<const uint4*>(p + j * 128);
                        vw[u][4 * j] = x.x;
                        vw[u][4 * j + 1] = x.y;
                        vw[u][4 * j + 2] = x.z;
                        vw[u][4 * j + 3] = x.w;
                    }
                }
            }
#pragma unroll
            for (int w = 0; w < C::VW; ++w) {
                const uint32_t r0 = vw[0][w], r1 = vw[1][w], r2 = vw[2][w], r3 = vw[3][w];
                if (E4M3) {
                    const uint32_t x = __byte_perm(r0, r1, 0x5140), y = __byte_perm(r2, r3, 0x5140);
                    mma_f16(acc[2 * w], lo_f16x2(x), hi_f16x2(x), lo_f16x2(y), hi_f16x2(y), pb[0], pb[1]);
                    const uint32_t x2 = __byte_perm(r0, r1, 0x7362), y2 = __byte_perm(r2, r3, 0x7362);
                    mma_f16(acc[2 * w + 1], lo_f16x2(x2), hi_f16x2(x2), lo_f16x2(y2), hi_f16x2(y2),
                            pb[0], pb[1]);
                } else {
                    const uint32_t a0 = __byte_perm(r0, r1, 0x5410), a1 = __byte_perm(r0, r1, 0x7632);
                    const uint32_t a2 = __byte_perm(r2, r3, 0x5410), a3 = __byte_perm(r2, r3, 0x7632);
                    mma_bf16(acc[w], a0, a1, a2, a3, pb[0], pb[1]);
                    mma_bf16(acc[w], a0, a1, a2, a3, pl[0], pl[1]);
                }
            }
        }
        slot = slot1;
        slot1 = slot_of(pos_s[(it & 1) * 32], page_s[0], tile + 2 * step);
    }

    // ---- merge: lanes, warps, CTAs ----
    ptx::cp_async_wait<0>();
    __syncwarp();                                       // the rings are free
    float* o_s = reinterpret_cast<float*>(smem);        // warp w's O^T at w * RING
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
        if (r8 == 0) {
            float* ml = ml_s + warp * 3 * PT_H + 2 * t4 + c;
            ml[0] = met ? m1[c] : PT_EMPTY;
            ml[PT_H] = E4M3 ? m2[c] : m1[c];
            ml[2 * PT_H] = l[c];
        }
    }
    // [row tile and half][head parity][head pair][r8]: no bank met twice
    {
        float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int j = 0; j < C::DT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mine[(2 * j + (i >> 1)) * 64 + (i & 1) * 32 + t4 * 8 + r8] = acc[j][i];
    }
    __syncthreads();
    // a thread: one (head, r8) and EPT consecutive dims
    const int combo = threadIdx.x & 63, part = threadIdx.x >> 6;
    const int h = 2 * (combo >> 3 & 3) + (combo >> 5);
    const int dr = combo & 7;
    const int dim = E4M3 ? dr * (D / 8) + part * C::EPT
                         : (C::EPT == 8 ? part * 64 + dr * 8 : dr * 8 + part * 4);
    float M1 = PT_EMPTY, M2 = PT_NONE, L = 0.f, o[C::EPT];
#pragma unroll
    for (int w = 0; w < PT_WARPS; ++w) {
        M1 = fmaxf(M1, ml_s[w * 3 * PT_H + h]);
        M2 = fmaxf(M2, ml_s[w * 3 * PT_H + PT_H + h]);
    }
#pragma unroll
    for (int i = 0; i < C::EPT; ++i) o[i] = 0.f;
#pragma unroll
    for (int w = 0; w < PT_WARPS; ++w) {
        const float* ml = ml_s + w * 3 * PT_H + h;
        const float f = ex2(ml[PT_H] - M2);
        L += ml[2 * PT_H] * ex2(ml[0] - M1);
        const float* src = o_s + w * (C::RING / 4) + part * C::EPT * 64 + combo;
#pragma unroll
        for (int i = 0; i < C::EPT; ++i) o[i] += f * src[i * 64];
    }
    // What takes a sum of weighted values from the reference m2 to m1, in two equal factors:
    // the scales of values alone reach from 2^-126 to 2^127, so that one would be flushed.
    auto lift = [](float x) { return E4M3 ? ex2(0.5f * x) : 1.f; };
    if (n_cta > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        // thread t's elements go to CTA t / tpc, place (source CTA, t % tpc)
        const uint32_t tpc = (PT_THREADS + n_cta - 1) / n_cta;
        const uint32_t to = threadIdx.x / tpc, at = threadIdx.x % tpc;
        const uint32_t dst = cluster_addr(recv, to) + 4 * C::EPT * (rank * tpc + at);
#pragma unroll
        for (int i = 0; i < C::EPT; i += 4) st_cluster4(dst + 4 * i, o + i);
        const uint32_t ml = cluster_addr(recv_ml, to) + 4 * (rank * 3 * PT_H + h);
        st_cluster(ml, M1);                             // (equal values from a head's threads)
        st_cluster(ml + 4 * PT_H, M2);
        st_cluster(ml + 8 * PT_H, L);
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                     ::: "memory");
    }
    if (n_cta == 1) {
        const bool empty = M1 == PT_EMPTY;
        const float f = 1.f / L, e = lift(M2 - M1);
        if (h < nh) {
            __nv_bfloat16* dst = a.O + (hbase + h) * D + dim;
            uint32_t w[C::EPT / 2];
#pragma unroll
            for (int i = 0; i < C::EPT / 2; ++i)
                w[i] = ptx::pack_bf16(empty ? 0.f : o[2 * i] * f * e * e,
                                      empty ? 0.f : o[2 * i + 1] * f * e * e);
            if (C::EPT == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
            if (a.lse && dim == 0)
                a.lse[hbase + h] = empty ? -INFINITY : (M1 + log2f(L)) * 0.6931471805599453f;
        }
        return;
    }
    // this CTA finishes the elements of threads rank * tpc .. of every CTA
    const uint32_t tpc = (PT_THREADS + n_cta - 1) / n_cta;
    const uint32_t own = min(tpc, PT_THREADS - min(rank * tpc, (uint32_t)PT_THREADS));
    for (uint32_t x = threadIdx.x; x < own * C::EPT; x += PT_THREADS) {
        const uint32_t t = rank * tpc + x / C::EPT, i = x % C::EPT;
        const int cb = t & 63, pt = t >> 6, hh = 2 * (cb >> 3 & 3) + (cb >> 5), rr = cb & 7;
        const int dd = (E4M3 ? rr * (D / 8) + pt * C::EPT
                             : (C::EPT == 8 ? pt * 64 + rr * 8 : rr * 8 + pt * 4)) + i;
        float N1 = PT_EMPTY, N2 = PT_NONE, S = 0.f, v = 0.f;
#pragma unroll 4
        for (uint32_t c = 0; c < n_cta; ++c) {
            N1 = fmaxf(N1, recv_ml[c * 3 * PT_H + hh]);
            N2 = fmaxf(N2, recv_ml[c * 3 * PT_H + PT_H + hh]);
        }
#pragma unroll 4
        for (uint32_t c = 0; c < n_cta; ++c) {
            const float* ml = recv_ml + c * 3 * PT_H + hh;
            S += ml[2 * PT_H] * ex2(ml[0] - N1);
            v += recv[c * tpc * C::EPT + x] * ex2(ml[PT_H] - N2);
        }
        if (hh < nh) {
            const bool empty = N1 == PT_EMPTY;
            const float e = lift(N2 - N1);
            a.O[(hbase + hh) * D + dd] = __float2bfloat16_rn(empty ? 0.f : v / S * e * e);
            if (a.lse && dd == 0)
                a.lse[hbase + hh] = empty ? -INFINITY : (N1 + log2f(S)) * 0.6931471805599453f;
        }
    }
}

// Clusters of c CTAs (2, 4, 8, 16) that the current device holds at once; 0 where it takes
// none.  What its GPCs have room for, which is less than its SMs' places: 31 of 16 with four
// CTAs on an SM, 21 with three.  Asked once per device.
template <bool E4M3, int D>
int cluster_room(int c)
{
    constexpr int MAXDEV = 64;
    static std::atomic<int> known[MAXDEV][PT_MAX_C + 1];   // one more than the answer
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < MAXDEV) {
        const int k = known[dev][c].load(std::memory_order_relaxed);
        if (k > 0) return k - 1;
    }
    const auto kern = paged_attn_kernel<E4M3, D>;
    cudaError_t e = ensure_smem_attr((const void*)kern, PagedCfg<E4M3, D>::BYTES);
    if (e == cudaSuccess && c > 8)
        e = cudaFuncSetAttribute((const void*)kern,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(PT_THREADS);
    cfg.dynamicSmemBytes = PagedCfg<E4M3, D>::BYTES;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)c;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    if (dev < MAXDEV) known[dev][c].store(n + 1, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_paged_attn(const lsa_paged_kv& kv, const void* Q, int64_t Nq, int Hq,
                              const int32_t* indices, const int32_t* counts, int s_max,
                              float scale, void* O, float* lse, cudaStream_t st)
{
    PagedAttnArgs a;
    a.Q = (const __nv_bfloat16*)Q;
    a.Nq = Nq;
    a.Hq = Hq;
    a.hpg = Hq / kv.Hkv;
    a.chunks = (a.hpg + PT_H - 1) / PT_H;
    a.indices = indices;
    a.counts = counts;
    a.s_max = s_max;
    a.page_shift = 0;
    while ((1 << a.page_shift) < kv.page) ++a.page_shift;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.O = (__nv_bfloat16*)O;
    a.lse = lse;
    const int64_t units = kv.B * Nq * kv.Hkv * a.chunks;
    const int64_t sms = sm_count(), slots = sms * (kv.format == LSA_KV_BF16 && kv.d == 128 ? 3 : 4);
    // CTAs per unit: those of the least cost by what was measured of 686 calls (2 to 512
    // units of 100 to 8,708 keys, heads of 64 and 128, both formats; the times are in
    // profiles/paged_split.csv), in tenths of a tile's
    // time: a warp's tiles, each dearer by a tenth for every CTA on the SM, and the merge
    // between CTAs, for every one on the SM.  On the mean it is within 1 % of the best
    // choice, where splits that fill half of the places were 4 % behind it (40 units of
    // 4,612 keys: 4 CTAs 18.9 us, 8 16.4; 128 units of 260 keys: one 6.3, two 8.8).
    // Clusters never fill the last places (148 units of 3,016 keys: 26.7 us with two, 35.1
    // with four, which the SMs' places would just hold), still less a second wave (256 bf16
    // units: 58.8 us with one, 75.1 with two; 32 units: 14.6 us with 8, 22.7 with 16, of which
    // the device holds 31).
    auto split = [&](int64_t n, auto room) {
        int best = 1;
        int64_t least = 0;
        for (int c = 1; c <= PT_MAX_C; c *= 2) {
            const int64_t ctas = n * c, on_sm = (ctas + sms - 1) / sms;
            if (c > 1 && (ctas * 20 > slots * 19 || n > room(c))) break;
            const int tiles = (int)(((int64_t)s_max + 32 * PT_WARPS * c - 1) / (32 * PT_WARPS * c));
            const int64_t merge = c == 1 ? 0 : c == 2 ? 22 : c < 16 ? 18 : 27;
            const int64_t cost = tiles * (10 + (on_sm < 4 ? on_sm : 4)) + merge * on_sm;
            if (c == 1 || cost < least) {
                best = c;
                least = cost;
            }
        }
        return best;
    };
    // Units past the last whole wave would run alone for as long as a full wave's.  Where
    // they fill less than 3/8 of one they follow in a launch of their own, split like a
    // small call's (502 bf16 units of 4,612 keys: 117 us in one launch, 101 in two; 446 of
    // them 114 against 91; 950 of them 191 against 178; 640 8-bit units of 2,564 keys 85
    // against 75, of 4,612 keys 145 against 122).  With more of them there is little to win
    // (700 bf16 units 149.5 against 154), nor with short rows (596 units of 260 keys 15.5
    // against 17.2; of 1,156 keys 41.0 against 40.7) or after three waves (1,840 units 183
    // against 184).  The second launch waits for the first one's end before it reads, as
    // everything that may read what an earlier kernel wrote: with rows of unequal length,
    // which fill the last wave by themselves, that wait is lost (640 units of 0 to 2,564
    // keys 42 us in one launch, 52 in two; 502 bf16 units of 0 to 4,612 keys 63 against
    // 76), but only the device knows their counts.
    const int64_t rest = units > slots && units < 3 * slots && s_max >= 1024 ? units % slots : 0;
    const int64_t behind = rest <= slots * 3 / 8 ? rest : 0;
    auto run = [&](auto kern, int bytes, auto room) {
        cudaError_t e = ensure_smem_attr((const void*)kern, bytes);
        if (e != cudaSuccess) return e;
        auto launch = [&](int64_t n) {
            const int c = split(n, room);
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(n * c));
            cfg.blockDim = dim3(PT_THREADS);
            cfg.dynamicSmemBytes = bytes;
            cfg.stream = st;
            cudaLaunchAttribute at[2] = {dependent_launch()};
            at[1].id = cudaLaunchAttributeClusterDimension;
            at[1].val.clusterDim.x = (unsigned)c;
            at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
            cfg.attrs = at;
            cfg.numAttrs = c > 1 ? 2 : 1;
            e = cudaLaunchKernelEx(&cfg, kern, kv, a);
            if (e == cudaSuccess) note_launch();
            return e;
        };
        a.unit0 = 0;
        e = launch(units - behind);
        if (e != cudaSuccess || behind == 0) return e;
        a.unit0 = units - behind;
        return launch(behind);
    };
    cudaError_t e;
    if (kv.format == LSA_KV_E4M3)
        e = kv.d == 64 ? run(paged_attn_kernel<true, 64>, PagedCfg<true, 64>::BYTES,
                             cluster_room<true, 64>)
                       : run(paged_attn_kernel<true, 128>, PagedCfg<true, 128>::BYTES,
                             cluster_room<true, 128>);
    else
        e = kv.d == 64 ? run(paged_attn_kernel<false, 64>, PagedCfg<false, 64>::BYTES,
                             cluster_room<false, 64>)
                       : run(paged_attn_kernel<false, 128>, PagedCfg<false, 128>::BYTES,
                             cluster_room<false, 128>);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lsa
