// k_paged_attn.cu -- softmax attention over listed positions of a paged cache.
//
// For query head h with KV head g: z_t = scale <q_h, sK_t k_t>, o_h = sum_t
// exp(z_t - lse) sV_t v_t, lse = ln sum_t exp(z_t) over the row's listed
// positions t, whose rows the page table locates (sK, sV: the scales of 8-bit
// pages, 1 for bf16).
//
// A CTA per (query row, KV head), the keys in tiles of 32 as fp32 in shared
// memory, the group's query heads eight at a time.
#include "paged.cuh"

namespace lsa {

constexpr int PT_THREADS = 128;
constexpr int PT_K = 32;     // keys per tile
constexpr int PT_H = 8;      // query heads per pass

template <bool E4M3, int D>
__global__ void __launch_bounds__(PT_THREADS) paged_attn_kernel(
    lsa_paged_kv kv, const __nv_bfloat16* Q, int64_t Nq, int Hq, const int32_t* indices,
    const int32_t* counts, int s_max, float scale, __nv_bfloat16* O, float* lse)
{
    __shared__ float q_s[PT_H][D];
    __shared__ float k_s[PT_K][D + 1];
    __shared__ float v_s[PT_K][D + 1];
    __shared__ float p_s[PT_H][PT_K];
    __shared__ float m_s[PT_H], l_s[PT_H], f_s[PT_H];
    __shared__ int64_t slot_s[PT_K];
    const int hpg = Hq / kv.Hkv;
    const int64_t row = blockIdx.x / kv.Hkv;
    const int g = blockIdx.x % kv.Hkv;
    const int64_t b = row / Nq;
    const int n = min(max(counts[row], 0), s_max);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int h0 = 0; h0 < hpg; h0 += PT_H) {
        const int nh = min(PT_H, hpg - h0);
        const int64_t hbase = row * Hq + (int64_t)g * hpg + h0;
        __syncthreads();
        for (int x = tid; x < nh * D; x += PT_THREADS)
            q_s[x / D][x % D] = __bfloat162float(Q[hbase * D + x]);
        if (tid < PT_H) {
            m_s[tid] = -INFINITY;
            l_s[tid] = 0.f;
        }
        float acc[PT_H * D / PT_THREADS];
        for (float& x : acc) x = 0.f;
        for (int k0 = 0; k0 < n; k0 += PT_K) {
            __syncthreads();
            if (tid < PT_K) {
                int64_t slot = -1;
                if (k0 + tid < n) {
                    const int32_t t = indices[row * s_max + k0 + tid];
                    const int32_t pg = page_of(kv, b, t);
                    if (pg >= 0) slot = (int64_t)pg * kv.page + (t & (kv.page - 1));
                }
                slot_s[tid] = slot;
            }
            __syncthreads();
            for (int x = tid; x < PT_K * D; x += PT_THREADS) {
                const int r = x / D, c = x % D;
                const int64_t slot = slot_s[r];
                float kx = 0.f, vx = 0.f;
                if (slot >= 0) {
                    const int64_t off = (slot * kv.Hkv + g) * D + c;
                    if (E4M3) {
                        const float* s = kv.scales + (slot / SCALE_BLOCK) * 2 * kv.Hkv + g;
                        kx = e4m3_value(((const uint8_t*)kv.K)[off]) * s[0];
                        vx = e4m3_value(((const uint8_t*)kv.V)[off]) * s[kv.Hkv];
                    } else {
                        kx = __bfloat162float(((const __nv_bfloat16*)kv.K)[off]);
                        vx = __bfloat162float(((const __nv_bfloat16*)kv.V)[off]);
                    }
                }
                k_s[r][c] = kx;
                v_s[r][c] = vx;
            }
            __syncthreads();
            // a warp per head: its 32 logits, the running maximum and sum
            for (int h = warp; h < nh; h += PT_THREADS / 32) {
                float z = 0.f;
                for (int c = 0; c < D; ++c) z = fmaf(q_s[h][c], k_s[lane][c], z);
                z = slot_s[lane] >= 0 ? z * scale : -INFINITY;
                float m = z;
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float was = m_s[h];
                m = fmaxf(m, was);
                const float ref = m == -INFINITY ? 0.f : m;
                const float p = expf(z - ref);
                float sum = p;
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                p_s[h][lane] = p;
                __syncwarp();
                if (lane == 0) {
                    const float f = expf(was - ref);
                    f_s[h] = f;
                    l_s[h] = l_s[h] * f + sum;
                    m_s[h] = m;
                }
            }
            __syncthreads();
            for (int x = tid, j = 0; x < nh * D; x += PT_THREADS, ++j) {
                const int h = x / D, c = x % D;
                float o = acc[j] * f_s[h];
                for (int r = 0; r < PT_K; ++r)
                    if (slot_s[r] >= 0) o = fmaf(p_s[h][r], v_s[r][c], o);
                acc[j] = o;
            }
        }
        __syncthreads();
        for (int x = tid, j = 0; x < nh * D; x += PT_THREADS, ++j) {
            const float l = l_s[x / D];
            O[hbase * D + x] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[j] / l);
        }
        if (lse && tid < nh) lse[hbase + tid] = m_s[tid] + logf(l_s[tid]);
    }
}

cudaError_t launch_paged_attn(const lsa_paged_kv& kv, const void* Q, int64_t Nq, int Hq,
                              const int32_t* indices, const int32_t* counts, int s_max,
                              float scale, void* O, float* lse, cudaStream_t st)
{
    const unsigned grid = (unsigned)(kv.B * Nq * kv.Hkv);
    auto run = [&](auto kern) {
        kern<<<grid, PT_THREADS, 0, st>>>(kv, (const __nv_bfloat16*)Q, Nq, Hq, indices, counts,
                                          s_max, scale, (__nv_bfloat16*)O, lse);
    };
    if (kv.format == LSA_KV_E4M3)
        kv.d == 64 ? run(paged_attn_kernel<true, 64>) : run(paged_attn_kernel<true, 128>);
    else
        kv.d == 64 ? run(paged_attn_kernel<false, 64>) : run(paged_attn_kernel<false, 128>);
    note_launch();
    return cudaGetLastError();
}

}  // namespace lsa
