// k_paged_append.cu -- new tokens' keys and values into a paged cache, keys
// (and the same tokens' queries) rotated by position on the way.
//
// Pair j of a head at position t turns by a = t * inv_freq[j]:
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a).
// 8-bit pages: a block of 16 slots and a head share a power-of-two scale s, the
// smallest whose 448-fold reaches the block's magnitudes; code = e4m3(x / s).
//
// Bound by memory: every value is read and written once.  A CTA takes 16
// consecutive positions (one scale block) of a sequence, so that a block's
// maximum never leaves it.  Its threads first turn positions into cosines and
// sines (one pair per token and frequency for all heads, in shared memory),
// then
//   * a warp takes a KV head's keys or values of all 16 tokens: D/16 lanes per
//     token, each holding two 16-byte chunks whose elements are the two halves
//     of its pairs; the scale is a maximum over the warp, no barrier;
//   * the queries go over (token, head) items, the token fixed for a group of
//     lanes, so that its cosines stay in registers over the heads; a block of
//     few new tokens (decode) spreads its heads over all groups instead.
// Positions are turned in double: t * inv_freq / 2 pi as a product with its
// rounding error kept, so that far positions lose nothing, reduced to an
// eighth of a turn before the fp32 sine and cosine.
#include "paged.cuh"

namespace lsa {

constexpr int PA_THREADS = 256;
constexpr int PA_WARPS = PA_THREADS / 32;

// cos and sin of 2 pi * (t * f / (2 pi)).
__device__ __forceinline__ void turn(int64_t t, float f, float* c, float* s)
{
    constexpr double INV = 0.15915494309189535, INV_LO = -9.839338337591243e-18;   // 1 / (2 pi)
    const double fd = (double)f, td = (double)t;
    const double p = fd * INV;
    const double pl = fma(fd, INV, -p) + fd * INV_LO;
    const double w = td * p;
    const double wl = fma(td, p, -w) + td * pl;
    const double r = (w - rint(w)) + wl;             // turns, about [-1/2, 1/2]
    const double q = rint(4.0 * r);
    float sn, cs;
    sincospif((float)(2.0 * (r - 0.25 * q)), &sn, &cs);
    const int k = (int)q;
    const float a = (k & 1) ? sn : cs, b = (k & 1) ? cs : sn;
    *c = ((k + 1) & 2) ? -a : a;
    *s = (k & 2) ? -b : b;
}

__device__ __forceinline__ void unpack8(float* x, const uint4& w)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float* x)
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Eight values times inv as codes.
__device__ __forceinline__ uint2 codes8(const float* x, float inv)
{
    uint32_t u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        u[i] = (uint32_t)e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) |
               (uint32_t)e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16;
    return make_uint2(u[0], u[1]);
}

// The cosines and sines of a lane's pairs, as rotate16 takes them.
struct Turns {
    float c[8], s[8];
};

// Turns a lane's two chunks.  Halves: pairs (lo[e], hi[e]).  Interleaved: pairs
// (2i, 2i + 1) of lo with turns 0 .. 3, of hi with turns 4 .. 7.
__device__ __forceinline__ void rotate16(float* lo, float* hi, const Turns& r, bool inter)
{
    if (inter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = lo[2 * i], y = lo[2 * i + 1], u = hi[2 * i], v = hi[2 * i + 1];
            lo[2 * i] = x * r.c[i] - y * r.s[i];
            lo[2 * i + 1] = y * r.c[i] + x * r.s[i];
            hi[2 * i] = u * r.c[4 + i] - v * r.s[4 + i];
            hi[2 * i + 1] = v * r.c[4 + i] + u * r.s[4 + i];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = lo[e], y = hi[e];
            lo[e] = x * r.c[e] - y * r.s[e];
            hi[e] = y * r.c[e] + x * r.s[e];
        }
    }
}

template <bool E4M3, int D>
__global__ void __launch_bounds__(PA_THREADS, 3) paged_append_kernel(lsa_paged_kv kv, AppendArgs a)
{
    constexpr int LPT = D / 16;              // lanes per token
    constexpr int TPW = 32 / LPT;            // tokens per warp and pass
    constexpr int NP = SCALE_BLOCK / TPW;    // passes over the block's tokens
    constexpr int GROUPS = PA_THREADS / LPT;
    constexpr int QB = 4;                    // query heads in flight per group
    __shared__ __align__(16) float cos_s[SCALE_BLOCK][D / 2], sin_s[SCALE_BLOCK][D / 2];
    const int64_t b = blockIdx.y;
    const int64_t start = a.start[b];
    int64_t n = a.n_new ? a.n_new[b] : a.Nq;
    if (n > a.Nq) n = a.Nq;
    if (n <= 0) return;
    if (start < 0) {
        if (blockIdx.x == 0 && threadIdx.x == 0) dev_error(kv.status, DEV_BAD_PAGE, (uint32_t)start);
        return;
    }
    const int64_t p0 = (start / SCALE_BLOCK + blockIdx.x) * SCALE_BLOCK;
    const int64_t end = start + n;
    // this call's tokens of the block: slots i0 .. i1 - 1
    const int i0 = (int)(p0 > start ? 0 : start - p0);
    const int i1 = (int)(end - p0 < SCALE_BLOCK ? end - p0 : SCALE_BLOCK);
    if (i0 >= i1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hkv = kv.Hkv;
    const int64_t row0 = b * a.Nq + (p0 - start);        // row of slot 0's token
    int32_t pg = -1;
    if (p0 < kv.max_pages * kv.page) {
        pg = kv.page_table[b * kv.max_pages + (p0 >> (__ffs(kv.page) - 1))];
        if (pg < 0 || pg >= kv.n_pages) pg = -1;
    }
    if (pg < 0 && threadIdx.x == 0) dev_error(kv.status, DEV_BAD_PAGE, (uint32_t)p0);

    // frequency f of a token at place pos(f): a lane's four or eight turns are
    // 16-byte runs, the runs of consecutive lanes side by side
    const int nf = a.rot / 2;
    const bool inter = a.interleaved != 0;
    for (int x = threadIdx.x; x < (i1 - i0) * nf; x += PA_THREADS) {
        const int i = i0 + x / nf, f = x % nf;
        const int at = inter ? f : ((f >> 2) & 1) * (nf / 2) + (f >> 3) * 4 + (f & 3);
        turn(p0 + i, a.inv_freq[f], &cos_s[i][at], &sin_s[i][at]);
    }
    __syncthreads();

    // a lane's chunks: of the r chunks that turn, (j, j + r/2); of the others
    // likewise
    const int j = lane % LPT;
    const int rh = a.rot / 16;                           // pairs of chunks that turn
    const bool turns = j < rh;
    const int ca = 8 * (turns ? j : j + rh);
    const int cb = ca + (turns ? 8 * rh : D / 2 - 8 * rh);
    auto load_turns = [&](Turns& r, int i) {
        const int at = inter ? 4 * (j + rh) : nf / 2 + 4 * j;
        *reinterpret_cast<float4*>(r.c) = *reinterpret_cast<const float4*>(&cos_s[i][4 * j]);
        *reinterpret_cast<float4*>(r.c + 4) = *reinterpret_cast<const float4*>(&cos_s[i][at]);
        *reinterpret_cast<float4*>(r.s) = *reinterpret_cast<const float4*>(&sin_s[i][4 * j]);
        *reinterpret_cast<float4*>(r.s + 4) = *reinterpret_cast<const float4*>(&sin_s[i][at]);
    };

    // ---- keys and values ----
    const int64_t slot0 = (int64_t)pg * kv.page + (p0 & (kv.page - 1));
    for (int it = warp; it < 2 * Hkv && pg >= 0; it += PA_WARPS) {
        const bool is_v = it >= Hkv;
        const int h = is_v ? it - Hkv : it;
        const __nv_bfloat16* src = (is_v ? a.v : a.k) + h * D;
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
        uint4 wa[NP], wb[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int i = p * TPW + lane / LPT;
            wa[p] = wb[p] = make_uint4(0u, 0u, 0u, 0u);
            if (i >= i0 && i < i1) {
                const __nv_bfloat16* r = src + (row0 + i) * stride;
                wa[p] = __ldcs(reinterpret_cast<const uint4*>(r + ca));
                wb[p] = __ldcs(reinterpret_cast<const uint4*>(r + cb));
            }
        }
        if (!E4M3) {
            __nv_bfloat16* pool = (__nv_bfloat16*)(is_v ? kv.V : kv.K) + h * D;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int i = p * TPW + lane / LPT;
                if (i < i0 || i >= i1) continue;
                if (!is_v && turns) {
                    float lo[8], hi[8];
                    Turns r;
                    load_turns(r, i);
                    unpack8(lo, wa[p]);
                    unpack8(hi, wb[p]);
                    rotate16(lo, hi, r, inter);
                    wa[p] = pack8(lo);
                    wb[p] = pack8(hi);
                }
                __nv_bfloat16* dst = pool + (slot0 + i) * Hkv * D;
                *reinterpret_cast<uint4*>(dst + ca) = wa[p];
                *reinterpret_cast<uint4*>(dst + cb) = wb[p];
            }
            continue;
        }
        float lo[NP][8], hi[NP][8];
        float amax = 0.f;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int i = p * TPW + lane / LPT;
            unpack8(lo[p], wa[p]);
            unpack8(hi[p], wb[p]);
            if (!is_v && turns && i >= i0 && i < i1) {
                Turns r;
                load_turns(r, i);
                rotate16(lo[p], hi[p], r, inter);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                amax = fmaxf(amax, fmaxf(finite_abs(lo[p][e]), finite_abs(hi[p][e])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        uint8_t* pool = (uint8_t*)(is_v ? kv.V : kv.K) + h * D;
        float* scale = kv.scales + ((slot0 / SCALE_BLOCK) * 2 + is_v) * Hkv + h;
        float s = e4m3_scale(amax);
        if (i0 > 0) {                        // the block held earlier tokens
            const float was = *scale;
            if (s > was) {
                const float f = was / s;
                for (int i = lane / LPT; i < i0; i += TPW) {
                    uint8_t* dst = pool + (slot0 + i) * Hkv * D;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint2* at = reinterpret_cast<uint2*>(dst + (u ? cb : ca));
                        const uint2 w = *at;
                        float x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            x[e] = e4m3_value((uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))));
                        *at = codes8(x, f);
                    }
                }
            } else {
                s = was;
            }
        }
        const float inv = 1.f / s;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int i = p * TPW + lane / LPT;
            if (i < i0 || i >= i1) continue;
            uint8_t* dst = pool + (slot0 + i) * Hkv * D;
            *reinterpret_cast<uint2*>(dst + ca) = codes8(lo[p], inv);
            *reinterpret_cast<uint2*>(dst + cb) = codes8(hi[p], inv);
        }
        __syncwarp();                        // every lane has read the old scale
        if (lane == 0) *scale = s;
    }

    // ---- queries: groups over (token, head), the token fixed ----
    if (a.Hq == 0) return;
    int tp = 1;                              // token slots, a power of two
    while (tp < i1 - i0) tp *= 2;
    const int grp = threadIdx.x / LPT;
    const int i = i0 + (grp & (tp - 1));
    const int hs = GROUPS / tp;
    if (i >= i1) return;
    Turns r;
    if (turns) load_turns(r, i);
    const __nv_bfloat16* src = a.q + (row0 + i) * a.q_stride;
    __nv_bfloat16* dst = a.q_out + (row0 + i) * (int64_t)a.Hq * D;
    for (int h0 = grp / tp; h0 < a.Hq; h0 += QB * hs) {
        uint4 wa[QB], wb[QB];
#pragma unroll
        for (int u = 0; u < QB; ++u) {
            const int h = h0 + u * hs;
            if (h < a.Hq) {
                wa[u] = __ldcs(reinterpret_cast<const uint4*>(src + h * D + ca));
                wb[u] = __ldcs(reinterpret_cast<const uint4*>(src + h * D + cb));
            }
        }
#pragma unroll
        for (int u = 0; u < QB; ++u) {
            const int h = h0 + u * hs;
            if (h < a.Hq) {
                if (turns) {
                    float lo[8], hi[8];
                    unpack8(lo, wa[u]);
                    unpack8(hi, wb[u]);
                    rotate16(lo, hi, r, inter);
                    wa[u] = pack8(lo);
                    wb[u] = pack8(hi);
                }
                *reinterpret_cast<uint4*>(dst + h * D + ca) = wa[u];
                *reinterpret_cast<uint4*>(dst + h * D + cb) = wb[u];
            }
        }
    }
}

cudaError_t launch_paged_append(const lsa_paged_kv& kv, const AppendArgs& a, cudaStream_t st)
{
    // Nq consecutive positions touch at most (Nq + 14) / 16 + 1 blocks
    const dim3 grid((unsigned)((a.Nq + SCALE_BLOCK - 2) / SCALE_BLOCK + 1), (unsigned)kv.B);
    auto run = [&](auto kern) { kern<<<grid, PA_THREADS, 0, st>>>(kv, a); };
    if (kv.format == LSA_KV_E4M3)
        kv.d == 64 ? run(paged_append_kernel<true, 64>) : run(paged_append_kernel<true, 128>);
    else
        kv.d == 64 ? run(paged_append_kernel<false, 64>) : run(paged_append_kernel<false, 128>);
    note_launch();
    return cudaGetLastError();
}

}  // namespace lsa
