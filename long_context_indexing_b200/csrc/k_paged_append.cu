// k_paged_append.cu -- new tokens' keys and values into a paged cache, keys
// (and the same tokens' queries) rotated by position on the way.
//
// Pair j of a head at position t turns by a = t * inv_freq[j]:
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a).
// 8-bit pages: a block of 16 slots and a head share a power-of-two scale s, the
// smallest whose 448-fold reaches the block's magnitudes; code = e4m3(x / s).
//
// A CTA per (sequence, block of 16 positions); a warp per head.
#include "paged.cuh"

namespace lsa {

constexpr int PA_THREADS = 128;

// Element c of head h of a token's row, rotated.
__device__ __forceinline__ float rotated(const __nv_bfloat16* row, int c, int rot, int inter,
                                         int64_t t, const float* inv_freq)
{
    const float x = __bfloat162float(row[c]);
    if (c >= rot) return x;
    const int half = rot / 2;
    const int j = inter ? c / 2 : (c < half ? c : c - half);
    const bool first = inter ? (c & 1) == 0 : c < half;
    const int o = inter ? c ^ 1 : (first ? c + half : c - half);
    const float y = __bfloat162float(row[o]);
    double sn, cs;
    sincos((double)t * (double)inv_freq[j], &sn, &cs);
    const float s = (float)sn, co = (float)cs;
    return first ? x * co - y * s : x * co + y * s;
}

template <bool E4M3>
__global__ void __launch_bounds__(PA_THREADS) paged_append_kernel(lsa_paged_kv kv, AppendArgs a)
{
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
    const int64_t t0 = p0 > start ? p0 : start;
    const int64_t t1 = p0 + SCALE_BLOCK < start + n ? p0 + SCALE_BLOCK : start + n;
    if (t0 >= t1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hkv = kv.Hkv, d = kv.d;
    __shared__ int32_t page_s;
    if (threadIdx.x == 0) page_s = page_of(kv, b, p0);
    __syncthreads();
    const int32_t pg = page_s;
    const int64_t base = (int64_t)pg * kv.page + (p0 & (kv.page - 1));   // slot of position p0
    const int64_t row0 = b * a.Nq - start;                               // + t: the token's row
    for (int it = warp; it < 2 * Hkv && pg >= 0; it += PA_THREADS / 32) {
        const int h = it >> 1;
        const bool is_v = it & 1;
        const __nv_bfloat16* src = (is_v ? a.v : a.k) + h * d;
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
        const int rot = is_v ? 0 : a.rot;
        if (!E4M3) {
            __nv_bfloat16* pool = (__nv_bfloat16*)(is_v ? kv.V : kv.K);
            for (int64_t t = t0; t < t1; ++t)
                for (int c = lane; c < d; c += 32)
                    pool[((base + t - p0) * Hkv + h) * d + c] = __float2bfloat16_rn(
                        rotated(src + (row0 + t) * stride, c, rot, a.interleaved, t, a.inv_freq));
            continue;
        }
        uint8_t* pool = (uint8_t*)(is_v ? kv.V : kv.K);
        float* scale = kv.scales + ((base / SCALE_BLOCK) * 2 + is_v) * Hkv + h;
        float amax = 0.f;
        for (int64_t t = t0; t < t1; ++t)
            for (int c = lane; c < d; c += 32)
                amax = fmaxf(amax, finite_abs(rotated(src + (row0 + t) * stride, c, rot,
                                                      a.interleaved, t, a.inv_freq)));
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float s = e4m3_scale(amax);
        if (t0 > p0) {                       // earlier tokens of the block
            const float was = *scale;
            if (s > was) {
                const float r = was / s;
                for (int64_t t = p0; t < t0; ++t)
                    for (int c = lane; c < d; c += 32) {
                        uint8_t* p = pool + ((base + t - p0) * Hkv + h) * d + c;
                        *p = (uint8_t)e4m3x2(e4m3_value(*p) * r, 0.f);
                    }
            } else {
                s = was;
            }
        }
        const float inv = 1.f / s;
        for (int64_t t = t0; t < t1; ++t)
            for (int c = lane; c < d; c += 32)
                pool[((base + t - p0) * Hkv + h) * d + c] = (uint8_t)e4m3x2(
                    rotated(src + (row0 + t) * stride, c, rot, a.interleaved, t, a.inv_freq) * inv,
                    0.f);
        __syncwarp();
        if (lane == 0) *scale = s;
    }
    // queries: a lane turns both elements of a pair (q_out may be q)
    for (int h = warp; h < a.Hq; h += PA_THREADS / 32)
        for (int64_t t = t0; t < t1; ++t) {
            const __nv_bfloat16* src = a.q + (row0 + t) * a.q_stride + h * d;
            __nv_bfloat16* dst = a.q_out + ((row0 + t) * a.Hq + h) * d;
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane + 32 * i < d)
                    x[i] = rotated(src, lane + 32 * i, a.rot, a.interleaved, t, a.inv_freq);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane + 32 * i < d) dst[lane + 32 * i] = __float2bfloat16_rn(x[i]);
            __syncwarp();
        }
}

cudaError_t launch_paged_append(const lsa_paged_kv& kv, const AppendArgs& a, cudaStream_t st)
{
    // Nq consecutive positions touch at most (Nq + 14) / 16 + 1 blocks
    const dim3 grid((unsigned)((a.Nq + SCALE_BLOCK - 2) / SCALE_BLOCK + 1), (unsigned)kv.B);
    if (kv.format == LSA_KV_E4M3)
        paged_append_kernel<true><<<grid, PA_THREADS, 0, st>>>(kv, a);
    else
        paged_append_kernel<false><<<grid, PA_THREADS, 0, st>>>(kv, a);
    note_launch();
    return cudaGetLastError();
}

}  // namespace lsa
