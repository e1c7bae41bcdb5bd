// paged.cuh -- declarations and device helpers of the paged KV cache (k_paged_append.cu,
// k_paged_attn.cu).
#pragma once

#include "lsa_internal.cuh"

namespace lsa {

constexpr int SCALE_BLOCK = 16;   // tokens that share an e4m3 scale
// status code beside those of DevErr: a position or page out of range
constexpr uint32_t DEV_BAD_PAGE = 5;

struct AppendArgs {
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    const __nv_bfloat16* q;      // nullable
    __nv_bfloat16* q_out;
    int64_t k_stride, v_stride, q_stride;
    int64_t Nq;
    int Hq;
    const int32_t* start;
    const int32_t* n_new;        // nullable
    const float* inv_freq;
    int rot;                     // rotated elements of a head
    int interleaved;
};
cudaError_t launch_paged_append(const lsa_paged_kv& kv, const AppendArgs& a, cudaStream_t st);
cudaError_t launch_paged_attn(const lsa_paged_kv& kv, const void* Q, int64_t Nq, int Hq,
                              const int32_t* indices, const int32_t* counts, int s_max,
                              float scale, void* O, float* lse, cudaStream_t st);

// Waits until the kernels that this one was launched behind have ended and their
// writes are visible.  What they may have written is read after it by ordinary loads and
// asynchronous copies only: a load through the read-only path (__ldg) says that its data
// does not change while the kernel lives, which it may before this wait, and the compiler
// may move such a load ahead of it.
__device__ __forceinline__ void grid_dependency()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The kernel is set up while the one before it on the stream still runs and waits
// for that one before it reads or writes anything (grid_dependency): calls in
// a row are 1 to 2 us closer (8 tokens' append 5.1 us a call against 3.1, a 33-row
// attention 10.2 against 8.1).  None lets a later call start before it ends: blocks
// that wait on an SM leave the next grid unevenly spread (64 rows in bf16 pages
// 52.0 us against 56.6 and more).
inline cudaLaunchAttribute dependent_launch()
{
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    return at;
}

// Smallest power of two 2^k, k >= -64, with amax <= 448 * 2^k (448 = 0.875 * 2^9).
__device__ __forceinline__ float e4m3_scale(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    int k = (int)(u >> 23) - 126 - 9 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (k < -64) k = -64;
    return __uint_as_float((uint32_t)(k + 127) << 23);
}

// Magnitude of a finite value, 0 for infinities and NaN.
__device__ __forceinline__ float finite_abs(float x)
{
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;
}

// Two codes (lo in the low byte), rounded to nearest even; infinities give the
// largest code, NaN stays NaN.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The values of two codes as f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t c)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

__device__ __forceinline__ float e4m3_value(uint8_t c)
{
    const uint32_t r = e4m3x2_f16x2((uint16_t)c);
    return __half2float(__ushort_as_half((unsigned short)(r & 0xffffu)));
}

}  // namespace lsa
