// kda_norm.cuh -- the norms around a mixer or block, fused with what stands next to them:
//   gated norm     out = x rsqrt(mean x^2 + eps) w act(z), or the gate before the norm
//   residual norm  r' = r + alpha ch act(z) n(x),  out = r' rsqrt(mean r'^2 + eps) w
// HBM-bound: every row is read once into registers, reduced there, and written once. A group of
// threads owns a row, eight channels per 16-byte access: up to 32 lanes (sums by shuffles) or a whole
// CTA (sums through shared memory). Groups walk the rows of a grid that fills the machine; with one or
// two vectors per thread the next row is loaded before the present one is reduced, with four a row's own
// loads are enough in flight. Sums and the norm are fp32.
// Residual norm of 32,768 x 2048, bf16 stream: 90 us (5.9 TB/s; a plain copy makes 6.7; arithmetic in pairs 92 us).
// Rows of one token's worth (128 x 2048 gated, 8 x 4096 residual) take 2.3 and 3.5 us, the chain of loads and sums.
#pragma once
#include "blk_common.cuh"

namespace kda {
namespace norm {

constexpr int WARP_THREADS = 128;  // CTA of the warp-group form
constexpr int CTA_THREADS = 512;   // most threads of the CTA form
constexpr int MAX_D = 16384;       // CTA_THREADS x 4 vectors of 8

// Eight channels at `at` of a tensor whose `rows` rows of `width` elements lie `stride` apart (the checked build looks)
__device__ __forceinline__ bool vec_ok(long long at, long long rows, long long stride, long long width)
{
    return gmem_ok(static_cast<size_t>(at), 8, static_cast<size_t>((rows - 1) * stride + width));
}

// Threads that share a row, and where this thread stands among them. CTA: the whole block, with
// two alternating rows of partial sums so that one barrier per sum is enough.
template <bool CTA>
struct Group {
    int tpr;                // threads per row
    int rank;
    float (*part)[32];
    int flip;
    __device__ __forceinline__ float sum(float v)
    {
        if constexpr (!CTA) {
            for (int m = tpr >> 1; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
            return v;
        } else {
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
            const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
            if (lane == 0) part[flip][threadIdx.x >> 5] = v;
            __syncthreads();
            v = lane < nw ? part[flip][lane] : 0.f;
            flip ^= 1;
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
            return v;
        }
    }
};

struct GatedParams {
    const uint16_t *x, *z;
    uint16_t *out;
    const float *w;
    long long xs, zs, os;   // elements between tokens
    long long rows;         // M * R
    int R, D, w_rows;
    float eps;
    int tpr;                // threads per row (warp-group form; a power of two)
};

// Instances by activation and gate order and arithmetic in pairs keep the issue slots free for the loads (32,768 x
// 16 rows of 128: 76.5 us with both as run-time choices and scalar arithmetic, 67.5 us so, 89 % of a plain copy); the
// one-vector form is held to 48 registers for ten CTAs per SM (seven: 69.6 us, twelve, which spill: 98.5 us).
template <int VPT, bool CTA, int ACT, bool FIRST>
__global__ void __launch_bounds__(CTA ? CTA_THREADS : WARP_THREADS, !CTA && VPT == 1 ? 10 : 1)
    kda_gated_norm_kernel(const GatedParams p)
{
    __shared__ float part[2][32];
    Group<CTA> gr{CTA ? static_cast<int>(blockDim.x) : p.tpr, CTA ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) & (p.tpr - 1), part, 0};
    const long long per = CTA ? 1 : WARP_THREADS / p.tpr, step = static_cast<long long>(gridDim.x) * per;
    const long long first = static_cast<long long>(blockIdx.x) * per + (CTA ? 0 : threadIdx.x / p.tpr);
    const float inv_d = 1.f / static_cast<float>(p.D);
    int c[VPT];
    bool live[VPT];
    float2 w[VPT][4];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        c[v] = 8 * (gr.rank + v * gr.tpr);
        live[v] = c[v] < p.D;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[v][i] = make_float2(1.f, 1.f);
        if (live[v] && p.w && p.w_rows == 1) blk::load8f(p.w + c[v], w[v]);
    }
    constexpr bool AHEAD = VPT <= 2;  // the next row is loaded before the present one is reduced
    uint4 xn[VPT], zn[VPT];
    // token and row of it, walked along without dividing
    const long long step_m = step / p.R;
    const int step_r = static_cast<int>(step - step_m * p.R);
    long long m = first / p.R, fm = m;
    int r = static_cast<int>(first - m * p.R), fr = r;
    auto advance = [&](long long &mm, int &rr) {
        mm += step_m;
        rr += step_r;
        if (rr >= p.R) {
            rr -= p.R;
            ++mm;
        }
    };
    const long long tokens = p.rows / p.R, width = static_cast<long long>(p.R) * p.D;
    auto fetch = [&](long long row, long long m, int r) {  // channels and rows that are not there count as zeros
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            xn[v] = zn[v] = make_uint4(0u, 0u, 0u, 0u);
            if (row < p.rows && live[v]) {
                const long long at = static_cast<long long>(r) * p.D + c[v];
                if (vec_ok(m * p.xs + at, tokens, p.xs, width)) xn[v] = *reinterpret_cast<const uint4 *>(p.x + m * p.xs + at);
                if (vec_ok(m * p.zs + at, tokens, p.zs, width)) zn[v] = *reinterpret_cast<const uint4 *>(p.z + m * p.zs + at);
            }
        }
    };
    if (AHEAD) fetch(first, fm, fr);
    // every group of a warp makes the same number of steps (the shuffles need all lanes)
    for (long long base = static_cast<long long>(blockIdx.x) * per; base < p.rows; base += step) {
        const long long row = base + (first - static_cast<long long>(blockIdx.x) * per);
        float2 x[VPT][4], z[VPT][4], ss = make_float2(0.f, 0.f);
        if (!AHEAD) fetch(row, m, r);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            blk::unpack8(xn[v], x[v]);
            blk::unpack8(zn[v], z[v]);
        }
        if (AHEAD) {
            advance(fm, fr);
            fetch(row + step, fm, fr);
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                z[v][i] = blk::apply_act2<ACT>(z[v][i]);
                if (FIRST) x[v][i] = fmul2(x[v][i], z[v][i]);
                ss = ffma2(x[v][i], x[v][i], ss);
            }
        const float inv = rsqrtf(fmaf(gr.sum(ss.x + ss.y), inv_d, p.eps));
        if (row < p.rows) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                if (!live[v]) continue;
                if (p.w && p.w_rows != 1) blk::load8f(p.w + static_cast<size_t>(r) * p.D + c[v], w[v]);
                float2 o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[i] = fmul2(fmul2(x[v][i], make_float2(inv, inv)), w[v][i]);
                    if (!FIRST) o[i] = fmul2(o[i], z[v][i]);
                }
                const long long at = m * p.os + static_cast<long long>(r) * p.D + c[v];
                if (vec_ok(at, tokens, p.os, width)) *reinterpret_cast<uint4 *>(p.out + at) = blk::pack8(o);
            }
        }
        advance(m, r);
    }
}

struct ResidualParams {
    const uint16_t *x, *z;
    const void *r;
    void *ro;
    uint16_t *out;
    const float *post, *chan, *w;
    long long xs, zs, rs, ros, os;
    long long rows;
    int D, act;
    float alpha, eps;
    int tpr;
};

// F32: the residual stream is fp32 (else bf16).
template <int VPT, bool CTA, bool F32>
__global__ void __launch_bounds__(CTA ? CTA_THREADS : WARP_THREADS) kda_residual_norm_kernel(const ResidualParams p)
{
    __shared__ float part[2][32];
    Group<CTA> gr{CTA ? static_cast<int>(blockDim.x) : p.tpr, CTA ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) & (p.tpr - 1), part, 0};
    const long long per = CTA ? 1 : WARP_THREADS / p.tpr, step = static_cast<long long>(gridDim.x) * per;
    const long long sub = CTA ? 0 : threadIdx.x / p.tpr;
    const float inv_d = 1.f / static_cast<float>(p.D);
    constexpr int RV = F32 ? 2 : 1;  // 16-byte vectors of eight residual channels
    int c[VPT];
    bool live[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        c[v] = 8 * (gr.rank + v * gr.tpr);
        live[v] = c[v] < p.D;
    }
    uint4 xn[VPT], zn[VPT], rn[VPT][RV];
    auto fetch = [&](long long row) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            xn[v] = zn[v] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < RV; ++k) rn[v][k] = make_uint4(0u, 0u, 0u, 0u);
            if (row < p.rows && live[v]) {
                if (vec_ok(row * p.xs + c[v], p.rows, p.xs, p.D)) xn[v] = *reinterpret_cast<const uint4 *>(p.x + row * p.xs + c[v]);
                if (p.z && vec_ok(row * p.zs + c[v], p.rows, p.zs, p.D)) zn[v] = *reinterpret_cast<const uint4 *>(p.z + row * p.zs + c[v]);
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.r) + (row * p.rs + c[v]) * (F32 ? 4 : 2));
                if (vec_ok(row * p.rs + c[v], p.rows, p.rs, p.D)) {
#pragma unroll
                    for (int k = 0; k < RV; ++k) rn[v][k] = src[k];
                }
            }
        }
    };
    constexpr bool AHEAD = VPT <= 2;
    if (AHEAD) fetch(static_cast<long long>(blockIdx.x) * per + sub);
    for (long long base = static_cast<long long>(blockIdx.x) * per; base < p.rows; base += step) {
        const long long row = base + sub;
        float x[VPT][8], r[VPT][8], ss = 0.f;
        if (!AHEAD) fetch(row);
        uint4 z[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            blk::unpack8(xn[v], x[v]);
            z[v] = zn[v];
            if constexpr (F32) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    r[v][4 * k] = __uint_as_float(rn[v][k].x);
                    r[v][4 * k + 1] = __uint_as_float(rn[v][k].y);
                    r[v][4 * k + 2] = __uint_as_float(rn[v][k].z);
                    r[v][4 * k + 3] = __uint_as_float(rn[v][k].w);
                }
            } else {
                blk::unpack8(rn[v][0], r[v]);
            }
        }
        if (AHEAD) fetch(row + step);
        if (p.post) {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[v][i], x[v][i], ss);
            const float inv = rsqrtf(fmaf(gr.sum(ss), inv_d, p.eps));
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                float w[8];
                if (live[v]) blk::load8f(p.post + c[v], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[v][i] = live[v] ? x[v][i] * inv * w[i] : 0.f;
            }
        }
        ss = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float ch[8], zf[8];
            if (p.chan && live[v]) blk::load8f(p.chan + c[v], ch);
            blk::unpack8(z[v], zf);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float u = x[v][i];
                if (p.z) u *= blk::apply_act(zf[i], p.act);
                if (p.chan) u *= ch[i];
                r[v][i] = live[v] ? fmaf(p.alpha, u, r[v][i]) : 0.f;
                ss = fmaf(r[v][i], r[v][i], ss);
            }
            if (p.ro && live[v] && row < p.rows && vec_ok(row * p.ros + c[v], p.rows, p.ros, p.D)) {
                if constexpr (F32) {
                    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.ro) + row * p.ros + c[v]);
                    dst[0] = make_float4(r[v][0], r[v][1], r[v][2], r[v][3]);
                    dst[1] = make_float4(r[v][4], r[v][5], r[v][6], r[v][7]);
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.ro) + row * p.ros + c[v]) = blk::pack8(r[v]);
                }
            }
        }
        if (!p.out) continue;
        const float inv = rsqrtf(fmaf(gr.sum(ss), inv_d, p.eps));
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!live[v] || row >= p.rows || !vec_ok(row * p.os + c[v], p.rows, p.os, p.D)) continue;
            float o[8], w[8];
            if (p.w) blk::load8f(p.w + c[v], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = p.w ? r[v][i] * inv * w[i] : r[v][i] * inv;
            *reinterpret_cast<uint4 *>(p.out + row * p.os + c[v]) = blk::pack8(o);
        }
    }
}

}  // namespace norm
}  // namespace kda
