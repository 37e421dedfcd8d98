// blk_common.cuh -- pieces shared by the operators around the mixer (convolution, state-space
// scan, norms): 8-channel bf16 vectors, the activations, varlen lookups.
#pragma once
#include "kda_common.cuh"

namespace kda {
namespace blk {

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + 2^(-z log2 e)). The exponential and the reciprocal are the hardware approximations. What counts is the
// rounding of the exponent, which has an ulp of 2^-17 for |z| above 44: the relative error is below 2^-20 for z > -22 and
// grows to about 2^-18 at z = -87, far under the bf16 rounding that follows. Below -87.3 the reciprocal is subnormal and
// comes out as 0, an error of less than 2^-126. z -> -inf gives 0, z -> +inf gives 1. The tanh form would lose the lower
// tail's relative precision.
__device__ __forceinline__ float sigmoid_fast(float z) { return rcp_approx(1.f + ex2_approx(-LOG2E * z)); }

__device__ __forceinline__ float apply_act(float z, int act)
{
    if (act == KDA_ACT_NONE) return z;
    const float s = sigmoid_fast(z);
    return act == KDA_ACT_SILU ? z * s : s;
}

// the same for pairs (paired multiply and add)
__device__ __forceinline__ float2 sigmoid_fast2(float2 z)
{
    const float2 u = fmul2(z, make_float2(-LOG2E, -LOG2E));
    const float2 v = fsub2(make_float2(ex2_approx(u.x), ex2_approx(u.y)), make_float2(-1.f, -1.f));
    return make_float2(rcp_approx(v.x), rcp_approx(v.y));
}

template <int ACT>
__device__ __forceinline__ float2 apply_act2(float2 z)
{
    if constexpr (ACT == KDA_ACT_NONE) return z;
    const float2 s = sigmoid_fast2(z);
    return ACT == KDA_ACT_SILU ? fmul2(z, s) : s;
}

// eight consecutive channels, as such or as four pairs
__device__ __forceinline__ void unpack8(const uint4 &w, float (&f)[8])
{
    f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
}
__device__ __forceinline__ void unpack8(const uint4 &w, float2 (&f)[4])
{
    f[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
    f[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
    f[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
    f[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4])
{
    return make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y), pack_bf16(f[3].x, f[3].y));
}
__device__ __forceinline__ void load8f(const float *p, float (&f)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ void load8f(const float *p, float2 (&f)[4])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y);
    f[3] = make_float2(b.z, b.w);
}

// Bounds of the packed sequence that holds token t: the last i with cu[i] <= t (for rising bounds
// that skips empty sequences). ok only where the bounds really enclose t inside [0, total].
struct Enclosing {
    int seq;
    long long b, e;
    bool ok;
};
__device__ __forceinline__ Enclosing find_sequence(const int64_t *cu, int nseq, long long total, long long t)
{
    int lo = 0, hi = nseq;
    while (hi - lo > 1) {
        const int mid = lo + ((hi - lo) >> 1);
        if (__ldg(cu + mid) <= t) lo = mid; else hi = mid;
    }
    const long long b = __ldg(cu + lo), e = __ldg(cu + lo + 1);
    return {lo, b, e, b >= 0 && b <= t && t < e && e <= total};
}

// One block looks every bound over: they rise from 0 to total, or the device error word says so.
__device__ __forceinline__ void check_bounds(const int64_t *cu, int nseq, long long total)
{
    bool bad = false;
    for (int i = threadIdx.x; i < nseq; i += blockDim.x) bad |= cu[i] > cu[i + 1];
    if (threadIdx.x == 0) bad |= cu[0] != 0 || cu[nseq] != total;
    if (bad) atomicOr(&g_dev_error, DEVERR_SEQLENS);
}

}  // namespace blk
}  // namespace kda
