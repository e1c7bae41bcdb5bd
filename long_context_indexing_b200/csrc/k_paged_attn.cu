// k_paged_attn.cu -- softmax attention over listed positions of a paged cache.
//
// For query head h with KV head g: z_t = scale <q_h, sK_t k_t>, o_h = sum_t
// exp(z_t - lse) sV_t v_t, lse = ln sum_t exp(z_t) over the row's listed
// positions t, whose rows the page table locates (sK, sV: the scales of 8-bit
// pages, 1 for bf16).
//
// A unit is (query row, KV head, up to 8 of its query heads); a cluster of C
// CTAs works on it, every warp of the cluster on tiles of KT keys of its own,
// and no warp waits for another until the end.  Keys are the M side of both
// products and the query heads the N side of 8, so that a group of 8 heads
// fills the warp MMA: S[key][head] = K Q^T, O^T[dim][head] += V^T P.
//   * K and V go from global memory straight into the MMA's A fragments: each
//     lane loads 16 consecutive bytes of a row and takes them as the fragment's
//     elements, which only renames the contraction index of K (Q's fragments
//     are renamed alike) and the output rows of V.  V's pairs along the keys
//     are byte permutations of two rows.  No shared memory, no barrier.
//   * 8-bit codes become f16, which holds them exactly; a query row is scaled
//     by a power of two so that f16 holds it too (what falls below f16's
//     subnormals is 2^-37 of the row's largest element).  sK multiplies the
//     logit in fp32; sV joins the exponent of the weight, w_t = 2^(z_t + log2
//     sV_t - m2), so that the f16 weight of the largest contribution is near 1
//     whatever the scales: 2^-11 relative.  The denominator sums 2^(z_t - m1)
//     in fp32 with a reference of its own.
//   * bf16 pages: the weight as the sum of two bf16 (2^-17 relative), since one
//     would add as much error as the output's rounding.
//   * The references m1, m2 move only when a value passes them by 2^8: one vote
//     per tile instead of a maximum over lanes.
// Warps, then the cluster's CTAs (through distributed shared memory) merge
// their (m1, m2, sum, O^T).
#include "paged.cuh"
#include "ptx.cuh"

namespace lsa {

constexpr int PT_WARPS = 4;
constexpr int PT_THREADS = 32 * PT_WARPS;
constexpr int PT_H = 8;             // query heads of a unit
constexpr float PT_NONE = -3e38f;   // reference before any key
constexpr float PT_SLACK = 8.f;     // log2 that a value may pass the reference by

template <bool E4M3, int D>
struct PagedCfg {
    static constexpr int ROWB = D * (E4M3 ? 1 : 2);   // bytes of one head's row
    // keys per tile: 64 registers of K and V in flight per lane at most
    static constexpr int KT = ROWB > 128 ? 16 : 32;
    static constexpr int MT = KT / 16;
    static constexpr int KW = ROWB / 16;              // words of a K row per lane
    static constexpr int VW = ROWB / 32;              // words of a V row per lane
    static constexpr int KS = D / 16;                 // contraction steps of S
    static constexpr int DT = D / 16;                 // row tiles of O^T
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
    __nv_bfloat16* O;
    float* lse;
};

__device__ __forceinline__ uint32_t ldg32(const void* p)
{
    uint32_t r;
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}
__device__ __forceinline__ void ldg128(uint32_t* r, const void* p)
{
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "l"(p));
}
__device__ __forceinline__ void ldg64(uint32_t* r, const void* p)
{
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "l"(p));
}
__device__ __forceinline__ void prefetch_l2(const void* p)
{
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void mma_f16_16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t lo_f16x2(uint32_t w) { return e4m3x2_f16x2((uint16_t)w); }
__device__ __forceinline__ uint32_t hi_f16x2(uint32_t w) { return e4m3x2_f16x2((uint16_t)(w >> 16)); }

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank)
{
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

template <bool E4M3, int D>
__global__ void __launch_bounds__(PT_THREADS, 3) paged_attn_kernel(lsa_paged_kv kv, PagedAttnArgs a)
{
    using C = PagedCfg<E4M3, D>;
    __shared__ float o_s[PT_WARPS][PT_H * D];
    __shared__ float m1_s[PT_WARPS][PT_H], m2_s[PT_WARPS][PT_H], l_s[PT_WARPS][PT_H];
    uint32_t rank, n_cta;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n_cta));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r8 = lane >> 2, t4 = lane & 3;
    const int64_t unit = blockIdx.x / n_cta;
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
    const int64_t t_end = kv.max_pages << a.page_shift;
    const int64_t tok_bytes = (int64_t)kv.Hkv * C::ROWB;
    const char* Kb = (const char*)kv.K + (int64_t)g * C::ROWB + t4 * 16;
    const char* Vb = (const char*)kv.V + (int64_t)g * C::ROWB + r8 * (E4M3 ? D / 8 : 16);

    const int n_tiles = (n + C::KT - 1) / C::KT;
    const int step = (int)n_cta * PT_WARPS;
    int tile = (int)rank * PT_WARPS + warp;

    // position of this lane's key of a tile (-2: none), its page, its slot (-1:
    // none).  A page is looked at one tile after its look-up.
    auto position = [&](int ti) {
        const int k = ti * C::KT + lane;
        return (lane < C::KT && k < n) ? __ldg(idx + k) : -2;
    };
    auto page = [&](int32_t t) {
        return (t >= 0 && t < t_end) ? __ldg(table + (t >> a.page_shift)) : -1;
    };
    auto slot_of = [&](int32_t t, int32_t pg) {
        if (t == -2) return -1;
        if (pg < 0 || pg >= kv.n_pages) {
            dev_error(kv.status, DEV_BAD_PAGE, (uint32_t)t);
            return -1;
        }
        return (pg << a.page_shift) + (t & (kv.page - 1));
    };

    uint32_t kw[C::MT][2][C::KW], vw[C::MT][4][C::VW];
    float ks = 0.f, vs = 0.f;                           // this lane's key's scales
    auto load_k = [&](int32_t slot, bool full) {
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int32_t s = __shfl_sync(0xffffffffu, slot, mt * 16 + u * 8 + r8);
                const char* p = Kb + s * tok_bytes;
#pragma unroll
                for (int j = 0; j < C::KW / 4; ++j) {
                    uint32_t* w = &kw[mt][u][4 * j];
                    if (full) {
                        ldg128(w, p + j * 64);
                    } else {
                        w[0] = w[1] = w[2] = w[3] = 0u;
                        if (s >= 0) ldg128(w, p + j * 64);
                    }
                }
            }
        if (E4M3) {
            ks = vs = 0.f;
            if (slot >= 0) {
                const float* s = kv.scales + (int64_t)(slot / SCALE_BLOCK) * (2 * kv.Hkv) + g;
                ks = __uint_as_float(ldg32(s));
                vs = __uint_as_float(ldg32(s + kv.Hkv));
            }
        }
    };
    auto load_v = [&](int32_t slot, bool full) {
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int32_t s =
                    __shfl_sync(0xffffffffu, slot, mt * 16 + (u >> 1) * 8 + 2 * t4 + (u & 1));
                const char* p = Vb + s * tok_bytes;
                uint32_t* w = vw[mt][u];
                if (!full) {
#pragma unroll
                    for (int j = 0; j < C::VW; ++j) w[j] = 0u;
                    if (s < 0) continue;
                }
                if (C::VW == 2) {
                    ldg64(w, p);
                } else {
#pragma unroll
                    for (int j = 0; j < C::VW / 4; ++j) ldg128(w + 4 * j, p + j * 128);
                }
            }
    };
    // a tile without gaps loads without predicates
    constexpr uint32_t FULL = C::KT == 32 ? 0xffffffffu : 0xffffu;
    auto load_tile_k = [&](int32_t slot, uint32_t valid) {
        if (valid == FULL) load_k(slot, true);
        else load_k(slot, false);
    };
    auto load_tile_v = [&](int32_t slot, uint32_t valid) {
        if (valid == FULL) load_v(slot, true);
        else load_v(slot, false);
    };

    // brings this lane's key's rows of a tile two ahead into L2
    auto prefetch = [&](int32_t slot) {
        if (slot < 0) return;
        const int64_t off = slot * tok_bytes + (int64_t)g * C::ROWB;
#pragma unroll
        for (int x = 0; x < C::ROWB; x += 128) {
            prefetch_l2((const char*)kv.K + off + x);
            prefetch_l2((const char*)kv.V + off + x);
        }
    };

    // the first tiles' positions and slots while the queries are read: in the
    // loop, slot is the tile's, slot1 and slot2 the next two tiles' (slot2's rows
    // on their way to L2), pos3 / pg3 and pos4 look two tiles further
    int32_t slot = -1, slot1 = -1, slot2 = -1, pos3 = -2, pg3 = -1, pos4 = -2;
    uint32_t valid = 0;
    if (tile < n_tiles) {
        const int32_t p0 = position(tile), p1 = position(tile + step), p2 = position(tile + 2 * step);
        pos3 = position(tile + 3 * step);
        pos4 = position(tile + 4 * step);
        const int32_t g0 = page(p0), g1 = page(p1), g2 = page(p2);
        pg3 = page(pos3);
        slot = slot_of(p0, g0);
        slot1 = slot_of(p1, g1);
        slot2 = slot_of(p2, g2);
        valid = __ballot_sync(0xffffffffu, slot >= 0);
        load_tile_k(slot, valid);
        load_tile_v(slot, valid);
        prefetch(slot1);
        prefetch(slot2);
    }

    // Q fragments: head r8; element order as K's lanes take their bytes
    uint32_t qb[C::KS][2];
    float cq[2];                                        // logit factor of heads 2 t4, 2 t4 + 1
    {
        float q[C::KS][4];
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < C::KS; ++s) {
            const int c = E4M3 ? (s / 4) * 64 + t4 * 16 + (s % 4) * 4
                               : (s / 2) * 32 + t4 * 8 + (s % 2) * 4;
            uint2 w = make_uint2(0u, 0u);
            if (r8 < nh) w = *reinterpret_cast<const uint2*>(a.Q + (hbase + r8) * D + c);
            if (!E4M3) {
                qb[s][0] = w.x;
                qb[s][1] = w.y;
            }
            q[s][0] = __uint_as_float(w.x << 16);
            q[s][1] = __uint_as_float(w.x & 0xffff0000u);
            q[s][2] = __uint_as_float(w.y << 16);
            q[s][3] = __uint_as_float(w.y & 0xffff0000u);
#pragma unroll
            for (int i = 0; i < 4; ++i) amax = fmaxf(amax, finite_abs(q[s][i]));
        }
        float f = a.scale_log2;
        if (E4M3) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // amax * 2^(13 - e) in [2^13, 2^14)
            const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100);
            const float up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
            f *= __uint_as_float((uint32_t)(e - 13 + 127) << 23);
#pragma unroll
            for (int s = 0; s < C::KS; ++s) {
                qb[s][0] = pack_f16(q[s][0] * up, q[s][1] * up);
                qb[s][1] = pack_f16(q[s][2] * up, q[s][3] * up);
            }
        }
        cq[0] = __shfl_sync(0xffffffffu, f, 8 * t4);
        cq[1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
    }

    float acc[C::DT][4];
#pragma unroll
    for (int j = 0; j < C::DT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    float m1[2] = {PT_NONE, PT_NONE}, m2[2] = {PT_NONE, PT_NONE}, l[2] = {0.f, 0.f};

    for (; tile < n_tiles; tile += step) {
        // ---- logits: keys mt*16 + r8 (+8), heads 2 t4 (+1) ----
        float z[C::MT][4];
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[mt][i] = 0.f;
#pragma unroll
            for (int s = 0; s < C::KS; ++s) {
                if (E4M3)
                    mma_f16_16816(z[mt], lo_f16x2(kw[mt][0][s]), lo_f16x2(kw[mt][1][s]),
                                  hi_f16x2(kw[mt][0][s]), hi_f16x2(kw[mt][1][s]), qb[s][0], qb[s][1]);
                else
                    ptx::mma_bf16_16816(z[mt], kw[mt][0][2 * s], kw[mt][1][2 * s],
                                        kw[mt][0][2 * s + 1], kw[mt][1][2 * s + 1], qb[s][0],
                                        qb[s][1]);
            }
        }
        float kf[C::MT][2], ev[C::MT][2];
        if (E4M3) {
            const float lv = __log2f(fmaxf(vs, 1e-37f));
#pragma unroll
            for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    kf[mt][u] = __shfl_sync(0xffffffffu, ks, mt * 16 + u * 8 + r8);
                    ev[mt][u] = __shfl_sync(0xffffffffu, lv, mt * 16 + u * 8 + r8);
                }
        }
        // the next tile's K and scales take the registers
        const uint32_t have = valid;
        slot = slot1;
        valid = __ballot_sync(0xffffffffu, slot >= 0);
        load_tile_k(slot, valid);

        bool over = false;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int u = i >> 1;
                z[mt][i] *= E4M3 ? kf[mt][u] * cq[i & 1] : cq[i & 1];
            }
        if (have != FULL) {
#pragma unroll
            for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!(have >> (mt * 16 + (i >> 1) * 8 + r8) & 1)) z[mt][i] = -INFINITY;
        }
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                over |= z[mt][i] > m1[i & 1] + PT_SLACK;
                if (E4M3) over |= z[mt][i] + ev[mt][i >> 1] > m2[i & 1] + PT_SLACK;
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x1 = m1[c], x2 = m2[c];
#pragma unroll
                for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        x1 = fmaxf(x1, z[mt][2 * u + c]);
                        if (E4M3) x2 = fmaxf(x2, z[mt][2 * u + c] + ev[mt][u]);
                    }
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) {
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
                    if (E4M3) x2 = fmaxf(x2, __shfl_xor_sync(0xffffffffu, x2, o));
                }
                if (!E4M3) x2 = x1;
                const float f2 = ex2(m2[c] - x2);
                l[c] *= ex2(m1[c] - x1);
                m1[c] = x1;
                m2[c] = x2;
#pragma unroll
                for (int j = 0; j < C::DT; ++j) {
                    acc[j][c] *= f2;
                    acc[j][c + 2] *= f2;
                }
            }
        }
        // ---- weights, transposed to (keys 2 t4, 2 t4 + 1; head r8) ----
        uint32_t pb[C::MT][2], pl[C::MT][2];
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float x0 = z[mt][2 * u], x1 = z[mt][2 * u + 1];
                const float p0 = ex2(x0 - m1[0]), p1 = ex2(x1 - m1[1]);
                l[0] += p0;
                l[1] += p1;
                if (E4M3) {
                    const float w0 = ex2(x0 + ev[mt][u] - m2[0]), w1 = ex2(x1 + ev[mt][u] - m2[1]);
                    pb[mt][u] = ptx::movmatrix_t(pack_f16(w0, w1));
                } else {
                    const uint32_t hi = ptx::pack_bf16(p0, p1);
                    const float e0 = p0 - __uint_as_float(hi << 16);
                    const float e1 = p1 - __uint_as_float(hi & 0xffff0000u);
                    pb[mt][u] = ptx::movmatrix_t(hi);
                    pl[mt][u] = ptx::movmatrix_t(ptx::pack_bf16(e0, e1));
                }
            }
        // ---- O^T += V^T P ----
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int w = 0; w < C::VW; ++w) {
                const uint32_t r0 = vw[mt][0][w], r1 = vw[mt][1][w];
                const uint32_t r2 = vw[mt][2][w], r3 = vw[mt][3][w];
                if (E4M3) {
                    const uint32_t x = __byte_perm(r0, r1, 0x5140), y = __byte_perm(r2, r3, 0x5140);
                    mma_f16_16816(acc[2 * w], lo_f16x2(x), hi_f16x2(x), lo_f16x2(y), hi_f16x2(y),
                                  pb[mt][0], pb[mt][1]);
                    const uint32_t x2 = __byte_perm(r0, r1, 0x7362), y2 = __byte_perm(r2, r3, 0x7362);
                    mma_f16_16816(acc[2 * w + 1], lo_f16x2(x2), hi_f16x2(x2), lo_f16x2(y2),
                                  hi_f16x2(y2), pb[mt][0], pb[mt][1]);
                } else {
                    const uint32_t a0 = __byte_perm(r0, r1, 0x5410), a1 = __byte_perm(r0, r1, 0x7632);
                    const uint32_t a2 = __byte_perm(r2, r3, 0x5410), a3 = __byte_perm(r2, r3, 0x7632);
                    ptx::mma_bf16_16816(acc[w], a0, a1, a2, a3, pb[mt][0], pb[mt][1]);
                    ptx::mma_bf16_16816(acc[w], a0, a1, a2, a3, pl[mt][0], pl[mt][1]);
                }
            }
        load_tile_v(slot, valid);
        slot1 = slot2;
        slot2 = slot_of(pos3, pg3);
        prefetch(slot2);
        pos3 = pos4;
        pg3 = page(pos3);
        pos4 = position(tile + 5 * step);
    }

    // ---- merge: lanes, warps, CTAs ----
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
        if (r8 == 0) {
            m1_s[warp][2 * t4 + c] = m1[c];
            m2_s[warp][2 * t4 + c] = E4M3 ? m2[c] : m1[c];
            l_s[warp][2 * t4 + c] = l[c];
        }
    }
#pragma unroll
    for (int j = 0; j < C::DT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // row tile j: dims of V's word j / 2 (8-bit) or j (bf16) of the lane
            const int dim = E4M3 ? r8 * (D / 8) + 2 * j + (i >> 1)
                                 : (j / 4) * 64 + r8 * 8 + 2 * (j % 4) + (i >> 1);
            o_s[warp][(2 * t4 + (i & 1)) * D + dim] = acc[j][i];
        }
    __syncthreads();
    // the CTA's warps into warp 0's arrays
    constexpr int EPT = PT_H * D / PT_THREADS;          // elements per thread, one head's
    {
        const int h = threadIdx.x * EPT / D;
        float M2 = m2_s[0][h];
#pragma unroll
        for (int w = 1; w < PT_WARPS; ++w) M2 = fmaxf(M2, m2_s[w][h]);
        float o[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) o[i] = 0.f;
#pragma unroll
        for (int w = 0; w < PT_WARPS; ++w) {
            const float f = ex2(m2_s[w][h] - M2);
#pragma unroll
            for (int i = 0; i < EPT; ++i) o[i] += f * o_s[w][threadIdx.x * EPT + i];
        }
        float M1 = PT_NONE, L = 0.f;
        if (threadIdx.x < PT_H) {
#pragma unroll
            for (int w = 0; w < PT_WARPS; ++w) M1 = fmaxf(M1, m1_s[w][threadIdx.x]);
#pragma unroll
            for (int w = 0; w < PT_WARPS; ++w)
                L += l_s[w][threadIdx.x] * ex2(m1_s[w][threadIdx.x] - M1);
        }
        __syncthreads();
        if (threadIdx.x < PT_H) {
            m1_s[0][threadIdx.x] = M1;
            l_s[0][threadIdx.x] = L;
        }
        if ((threadIdx.x * EPT) % D == 0) m2_s[0][h] = M2;
#pragma unroll
        for (int i = 0; i < EPT; ++i) o_s[0][threadIdx.x * EPT + i] = o[i];
    }
    if (n_cta > 1) cluster_sync();
    else __syncthreads();
    // the cluster's CTAs share the output's elements
    const int total = nh * D;
    for (int x = (int)rank * PT_THREADS + threadIdx.x; x < total; x += (int)n_cta * PT_THREADS) {
        const int h = x / D;
        float M1 = PT_NONE, M2 = PT_NONE, L = 0.f, o = 0.f;
        for (uint32_t c = 0; c < n_cta; ++c) {
            M1 = fmaxf(M1, ld_cluster(&m1_s[0][h], c));
            M2 = fmaxf(M2, ld_cluster(&m2_s[0][h], c));
        }
        for (uint32_t c = 0; c < n_cta; ++c) {
            L += ld_cluster(&l_s[0][h], c) * ex2(ld_cluster(&m1_s[0][h], c) - M1);
            o += ld_cluster(&o_s[0][x], c) * ex2(ld_cluster(&m2_s[0][h], c) - M2);
        }
        o = L == 0.f ? 0.f : o / L * ex2(M2 - M1);
        a.O[hbase * D + x] = __float2bfloat16_rn(o);
        if (a.lse && x % D == 0)
            a.lse[hbase + h] = L == 0.f ? -INFINITY : (M1 + log2f(L)) * 0.6931471805599453f;
    }
    if (n_cta > 1) cluster_sync();       // no CTA leaves while another reads its arrays
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
    // CTAs per unit: enough to fill the SMs three times over, each with at
    // least a tile per warp
    int c = 1;
    while (c < 8 && units * c * 2 <= 3 * 148 && s_max >= 2 * c * PT_WARPS * 32) c *= 2;
    auto run = [&](auto kern) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(units * c));
        cfg.blockDim = dim3(PT_THREADS);
        cfg.stream = st;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = (unsigned)c;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kern, kv, a);
    };
    cudaError_t e;
    if (kv.format == LSA_KV_E4M3)
        e = kv.d == 64 ? run(paged_attn_kernel<true, 64>) : run(paged_attn_kernel<true, 128>);
    else
        e = kv.d == 64 ? run(paged_attn_kernel<false, 64>) : run(paged_attn_kernel<false, 128>);
    if (e != cudaSuccess) return e;
    note_launch();
    return cudaGetLastError();
}

}  // namespace lsa
