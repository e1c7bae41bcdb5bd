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
// Positions are turned in 64-bit fixed point, so that far positions lose nothing,
// reduced to an eighth of a turn before the fp32 series.
//
// Rows come by 16-byte asynchronous copies into the lane's own places in shared
// memory (the first item while positions are turned, query heads four ahead), which
// leaves the registers to three CTAs per SM: with four CTAs the queries' part spills
// (heads of 64: padded batch 12.1 us against 11.7; 32,768 tokens 53 against 55), with
// two the keys' part waits (32,768 tokens of 4 heads 45 us against 38).
// Measured (B200): 32,768 tokens of 32/4 heads of 128 into 8-bit pages 101 us (637.6
// MB, 6.3 TB/s, 0.96 of a copy's rate: HBM); 2 x 4,096 tokens of 16/2 heads into
// bf16 pages 16.2 us (5.2 TB/s; 514 blocks, the queries in CTAs of their own); 7 padded
// prompts of up to 1,021 tokens of 24/8 heads of 64 10 us (waves of latencies:
// start 1.0 us, page and turns 2, keys and values 3.6, queries 2.8); 256 tokens of 32/4 heads 4.2 us, 8 tokens 3.1.
#include "paged.cuh"
#include "ptx.cuh"

namespace lsa {

constexpr int PA_THREADS = 256;
constexpr int PA_WARPS = PA_THREADS / 32;

// f / (2 pi) turns per position as a 64-bit fraction of a turn: a position's turn
// is then a product modulo 2^64, exact but for f's own rounding (2^-63 for |f| up to
// 2^44, so 2^-32 of a turn at the last position; past 2^53 the quotient's low part has
// whole turns and no fraction is left).
__device__ __forceinline__ uint64_t turns_of(float f)
{
    constexpr double INV = 0.15915494309189535, INV_LO = -9.839338337591243e-18;   // 1 / (2 pi)
    const double fd = (double)f;
    const double p = fd * INV;
    const double pl = fma(fd, INV, -p) + fd * INV_LO;
    return (uint64_t)__double2ll_rn((p - rint(p)) * 18446744073709551616.0) +
           (uint64_t)__double2ll_rn(pl * 18446744073709551616.0);
}

// cos and sin of position t's angle: the nearest quarter turn, and the Taylor
// series of the rest, |x| <= pi / 4 (sine to x^9, cosine to x^10: 2e-9 and less).
__device__ __forceinline__ void turn(uint32_t t, uint64_t f, float* c, float* s)
{
    const uint64_t a = f * t;
    const uint32_t k = (uint32_t)((a + (1ull << 61)) >> 62);
    const float x = (float)(int32_t)((uint32_t)(a >> 32) - (k << 30)) * 1.46291807926715968e-9f;
    const float y = x * x;                               // (2 pi / 2^32 above)
    float sn = fmaf(y, 2.75573192e-6f, -1.98412698e-4f);
    sn = fmaf(y, sn, 8.33333333e-3f);
    sn = fmaf(y, sn, -1.66666667e-1f);
    sn = fmaf(x * y, sn, x);
    float cs = fmaf(y, -2.75573192e-7f, 2.48015873e-5f);
    cs = fmaf(y, cs, -1.38888889e-3f);
    cs = fmaf(y, cs, 4.16666667e-2f);
    cs = fmaf(y, cs, -0.5f);
    cs = fmaf(y, cs, 1.f);
    const float u = (k & 1) ? sn : cs, v = (k & 1) ? cs : sn;
    *c = ((k + 1) & 2) ? -u : u;
    *s = (k & 2) ? -v : v;
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
    // (rows 64 bytes apart modulo 128 where two tokens' reads meet)
    constexpr int TURN_ROW = D / 2 + (D == 64 ? 16 : 0);
    __shared__ __align__(16) float cos_s[SCALE_BLOCK][TURN_ROW], sin_s[SCALE_BLOCK][TURN_ROW];
    __shared__ uint4 raw_s[PA_WARPS][QB][2][32];         // what a lane reads, NP or QB pairs
    grid_dependency();
    // one CTA for a block's keys, values and queries; or one for the queries and then one
    // for the rest; or one for the rest and several for the queries' heads
    const int parts = max((int)gridDim.z - 1, 1);        // of the queries
    const int kv_z = gridDim.z == 2 ? 1 : 0;
    const bool do_kv = (int)blockIdx.z == kv_z, do_q = a.Hq > 0 && (gridDim.z == 1 || !do_kv);
    const int64_t b = blockIdx.y;
    const int64_t start = a.start[b];
    int64_t n = a.n_new ? a.n_new[b] : a.Nq;
    if (n > a.Nq) n = a.Nq;
    if (n <= 0) return;
    if (start < 0) {                         // left out: queries of zeros, unless in place
        if (blockIdx.x == 0 && threadIdx.x == 0 && do_kv)
            dev_error(kv.status, DEV_BAD_PAGE, (uint32_t)start);
        if (do_q && a.q_out != a.q) {
            const int64_t part = gridDim.z > 2 ? (int)blockIdx.z - 1 : 0;
            uint4* dst = reinterpret_cast<uint4*>(a.q_out + b * a.Nq * a.Hq * D);
            for (int64_t i = (blockIdx.x * parts + part) * PA_THREADS + threadIdx.x;
                 i < n * a.Hq * (D / 8); i += (int64_t)gridDim.x * parts * PA_THREADS)
                dst[i] = make_uint4(0u, 0u, 0u, 0u);
        }
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
    if (pg < 0 && threadIdx.x == 0 && do_kv) dev_error(kv.status, DEV_BAD_PAGE, (uint32_t)p0);

    const int nf = a.rot / 2;
    const bool inter = a.interleaved != 0;
    // a lane's chunks: of the r chunks that turn, (j, j + r/2); of the others
    // likewise
    const int j = lane % LPT;
    const int rh = a.rot / 16;                           // pairs of chunks that turn
    const bool turns = j < rh;
    const int ca = 8 * (turns ? j : j + rh);
    const int cb = ca + (turns ? 8 * rh : D / 2 - 8 * rh);
    // ---- a KV head's keys or values of the block, each lane's own chunks; the
    // first of a warp is on its way while positions are turned ----
    constexpr int KB = QB / NP;                          // items that raw_s holds
    auto ask = [&](int it, int at) {
        const bool is_v = it >= Hkv;
        const __nv_bfloat16* src = (is_v ? a.v : a.k) + (is_v ? it - Hkv : it) * D;
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int i = p * TPW + lane / LPT;
            if (i >= i0 && i < i1) {
                const __nv_bfloat16* r = src + (row0 + i) * stride;
                ptx::cp_async16(&raw_s[warp][at + p][0][lane], r + ca);
                ptx::cp_async16(&raw_s[warp][at + p][1][lane], r + cb);
            }
        }
        ptx::cp_async_commit();
    };
    if (do_kv && warp < 2 * Hkv) ask(warp, 0);
    // queries: a group's token and heads
    int tp = 1;                              // token slots, a power of two
    while (tp < i1 - i0) tp *= 2;
    const int grp = threadIdx.x / LPT;
    const int i = i0 + (grp & (tp - 1));
    const int hs = GROUPS / tp * parts;
    const int h_first = grp / tp + (gridDim.z > 2 ? (int)blockIdx.z - 1 : 0) * (GROUPS / tp);
    auto ask_head = [&](int u, int h) {
        const __nv_bfloat16* src = a.q + (row0 + i) * a.q_stride;
        if (h < a.Hq) {
            ptx::cp_async16(&raw_s[warp][u][0][lane], src + h * D + ca);
            ptx::cp_async16(&raw_s[warp][u][1][lane], src + h * D + cb);
        }
        ptx::cp_async_commit();
    };
    auto ask_first = [&] {
#pragma unroll
        for (int u = 0; u < QB; ++u) ask_head(u, h_first + u * hs);
    };
    if (!do_kv && i < i1) ask_first();

    // frequency f of a token at place pos(f): a lane's four or eight turns are
    // 16-byte runs, the runs of consecutive lanes side by side
    {
        int fp = 8;                                      // frequencies, a power of two
        while (fp < nf) fp *= 2;
        const int f = threadIdx.x & (fp - 1);
        if (f < nf) {
            const uint64_t per = turns_of(a.inv_freq[f]);
            const int at = inter ? f : ((f >> 2) & 1) * (nf / 2) + (f >> 3) * 4 + (f & 3);
            for (int i = i0 + threadIdx.x / fp; i < i1; i += PA_THREADS / fp)
                turn((uint32_t)(p0 + i), per, &cos_s[i][at], &sin_s[i][at]);
        }
    }
    __syncthreads();

    auto load_turns = [&](Turns& r, int i) {
        const int at = inter ? 4 * (j + rh) : nf / 2 + 4 * j;
        *reinterpret_cast<float4*>(r.c) = *reinterpret_cast<const float4*>(&cos_s[i][4 * j]);
        *reinterpret_cast<float4*>(r.c + 4) = *reinterpret_cast<const float4*>(&cos_s[i][at]);
        *reinterpret_cast<float4*>(r.s) = *reinterpret_cast<const float4*>(&sin_s[i][4 * j]);
        *reinterpret_cast<float4*>(r.s + 4) = *reinterpret_cast<const float4*>(&sin_s[i][at]);
    };

    // ---- keys and values ----
    if (pg < 0) ptx::cp_async_wait<0>();     // (what was asked for is not used)
    const int64_t slot0 = (int64_t)pg * kv.page + (p0 & (kv.page - 1));
    int at = 0;
    for (int it = warp; it < 2 * Hkv && do_kv && pg >= 0; it += PA_WARPS) {
        const bool is_v = it >= Hkv;
        const int h = is_v ? it - Hkv : it;
        const int here = at;
        if (KB == 2) {                                   // the next item beside this one
            at = NP - at;
            if (it + PA_WARPS < 2 * Hkv) ask(it + PA_WARPS, at);
            else ptx::cp_async_commit();
            ptx::cp_async_wait<1>();
        } else {
            if (it != warp) ask(it, 0);
            ptx::cp_async_wait<0>();
        }
        // slot i's values of this lane, rotated
        auto values = [&](int p, int i, float* lo, float* hi) {
            unpack8(lo, raw_s[warp][here + p][0][lane]);
            unpack8(hi, raw_s[warp][here + p][1][lane]);
            if (!is_v && turns) {
                Turns r;
                load_turns(r, i);
                rotate16(lo, hi, r, inter);
            }
        };
        if (!E4M3) {
            __nv_bfloat16* pool = (__nv_bfloat16*)(is_v ? kv.V : kv.K) + h * D;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int i = p * TPW + lane / LPT;
                if (i < i0 || i >= i1) continue;
                float lo[8], hi[8];
                values(p, i, lo, hi);
                __nv_bfloat16* dst = pool + (slot0 + i) * Hkv * D;
                *reinterpret_cast<uint4*>(dst + ca) = pack8(lo);
                *reinterpret_cast<uint4*>(dst + cb) = pack8(hi);
            }
            continue;
        }
        // (keys are turned twice, for the maximum and for the codes: held, they would
        // cost half of the resident CTAs)
        float amax = 0.f;
        if (is_v) {
            __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);   // (passes NaN over)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int i = p * TPW + lane / LPT;
                if (i < i0 || i >= i1) continue;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint4 w = raw_s[warp][here + p][u][lane];
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x[e])));
                }
            }
            amax = fmaxf(__low2float(m), __high2float(m));
        } else {
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int i = p * TPW + lane / LPT;
                if (i < i0 || i >= i1) continue;
                float x[2][8];
                values(p, i, x[0], x[1]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    amax = fmaxf(amax, fmaxf(fabsf(x[0][e]), fabsf(x[1][e])));
            }
        }
        if (__any_sync(0xffffffffu, isinf(amax))) {      // the largest finite one instead
            amax = 0.f;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int i = p * TPW + lane / LPT;
                if (i < i0 || i >= i1) continue;
                float lo[8], hi[8];
                values(p, i, lo, hi);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    amax = fmaxf(amax, fmaxf(finite_abs(lo[e]), finite_abs(hi[e])));
            }
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
            float x[2][8];
            values(p, i, x[0], x[1]);
            *reinterpret_cast<uint2*>(dst + ca) = codes8(x[0], inv);
            *reinterpret_cast<uint2*>(dst + cb) = codes8(x[1], inv);
        }
        __syncwarp();                        // every lane has read the old scale
        if (lane == 0) *scale = s;
    }

    // ---- queries: groups over (token, head), the token fixed ----
    if (!do_q || i >= i1) return;
    Turns r;
    if (turns) load_turns(r, i);
    __nv_bfloat16* dst = a.q_out + (row0 + i) * (int64_t)a.Hq * D;
    if (do_kv) {                             // (raw_s held keys and values)
        ptx::cp_async_wait<0>();
        ask_first();
    }
    int h = h_first;
    for (int u = 0; h < a.Hq; h += hs, u = u + 1 < QB ? u + 1 : 0) {
        ptx::cp_async_wait<QB - 1>();
        uint4 xa = raw_s[warp][u][0][lane], xb = raw_s[warp][u][1][lane];
        ask_head(u, h + QB * hs);
        if (turns) {
            float lo[8], hi[8];
            unpack8(lo, xa);
            unpack8(hi, xb);
            rotate16(lo, hi, r, inter);
            xa = pack8(lo);
            xb = pack8(hi);
        }
        *reinterpret_cast<uint4*>(dst + h * D + ca) = xa;
        *reinterpret_cast<uint4*>(dst + h * D + cb) = xb;
    }
}

cudaError_t launch_paged_append(const lsa_paged_kv& kv, const AppendArgs& a, cudaStream_t st)
{
    // Nq consecutive positions touch at most (Nq + 14) / 16 + 1 blocks
    const int64_t blocks = (a.Nq + SCALE_BLOCK - 2) / SCALE_BLOCK + 1;
    // Up to two waves of blocks, the queries get CTAs of their own (8 tokens 4.2 us against
    // 3.5; past that the turns computed twice cost more than the shorter CTAs bring:
    // 16,384 tokens 53.7 us against 54.8), and while all CTAs come to two on an SM at most
    // their heads are cut into as many parts as one CTA's loads in flight make (256 tokens
    // 5.8 us against 4.2; with three on an SM 1,024 tokens 5.1 against 5.7).  With one part
    // the queries' CTAs are first, for they are the longer ones (2 x 4,096 tokens 17.6 us
    // against 16.2); with several the keys' and values' are.
    const int64_t ctas = blocks * kv.B, sms = sm_count();
    int parts = 0;
    if (a.Hq > 0 && ctas <= 2 * 3 * sms) {
        int tp = 1;                                      // tokens of a block at most
        while (tp < SCALE_BLOCK && tp < a.Nq) tp *= 2;
        const int batch = PA_THREADS * 16 / kv.d / tp * 4;     // heads a CTA has in flight
        const int64_t most = (a.Hq + batch - 1) / batch, fit = 2 * sms / ctas - 1;
        parts = (int)(fit < 1 ? 1 : fit < most ? fit : most);
    }
    const dim3 grid((unsigned)blocks, (unsigned)kv.B, 1u + parts);
    auto run = [&](auto kern) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(PA_THREADS);
        cfg.stream = st;
        cudaLaunchAttribute at = dependent_launch();
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kern, kv, a);
    };
    cudaError_t e;
    if (kv.format == LSA_KV_E4M3)
        e = kv.d == 64 ? run(paged_append_kernel<true, 64>) : run(paged_append_kernel<true, 128>);
    else
        e = kv.d == 64 ? run(paged_append_kernel<false, 64>) : run(paged_append_kernel<false, 128>);
    if (e != cudaSuccess) return e;
    note_launch();
    return cudaGetLastError();
}

}  // namespace lsa
