// kda_attn.cuh -- softmax attention of one new token per sequence over a paged cache of keys and values.
//   out = softmax(scale q K^T) V over the cached positions 0 .. position
// Simple form: a warp per (sequence, query head), D / 32 channels per lane, one pass over the cache with the running
// maximum and sum of the softmax.
#pragma once
#include "kda_rope.cuh"

namespace kda {
namespace attn {

using rope::Pages;

constexpr int THREADS = 128;

struct AttnParams {
    const uint16_t *q, *kc, *vc;
    uint16_t *out;
    float *lse;                 // [S, H] or NULL
    long long qs, os;           // elements between sequences
    const int64_t *positions;   // of the new tokens
    Pages pages;
    float scale;
    int S, H, HK, D;
};

// Cached tokens that a sequence's new token sees.
__device__ __forceinline__ long long tokens_of(const AttnParams &p, int seq)
{
    const int64_t pos = __ldg(p.positions + seq);
    if (pos < 0) return 0;
    if ((pos >> p.pages.shift) >= p.pages.width) {
        atomicOr(&g_dev_error, DEVERR_PAGES);
        return 0;
    }
    return pos + 1;
}

__global__ void __launch_bounds__(THREADS) kda_attn_step_kernel(const AttnParams p)
{
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
    if (w >= static_cast<long long>(p.S) * p.H) return;
    const int seq = static_cast<int>(w / p.H), h = static_cast<int>(w % p.H), hk = h / (p.H / p.HK), per = p.D / 32;
    const long long n = tokens_of(p, seq), page_size = 1LL << p.pages.shift;
    float q[4] = {}, acc[4] = {}, top = -INFINITY, sum = 0.f;
    for (int i = 0; i < per; ++i) q[i] = p.scale * __uint_as_float(static_cast<uint32_t>(p.q[seq * p.qs + h * p.D + per * lane + i]) << 16);
    for (long long t = 0; t < n; ++t) {
        const int page = __ldg(p.pages.table + static_cast<long long>(seq) * p.pages.width + (t >> p.pages.shift));
        if (page < 0 || page >= p.pages.count) {
            if (lane == 0) atomicOr(&g_dev_error, DEVERR_PAGES);
            continue;
        }
        const long long at = page * p.pages.stride + (hk * page_size + (t & (page_size - 1))) * p.D + per * lane;
        float x = 0.f;
        for (int i = 0; i < per; ++i) x = fmaf(q[i], __uint_as_float(static_cast<uint32_t>(p.kc[at + i]) << 16), x);
        for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
        const float hi = fmaxf(top, x), keep = expf(top - hi), e = expf(x - hi);
        top = hi;
        sum = sum * keep + e;
        for (int i = 0; i < per; ++i) acc[i] = acc[i] * keep + e * __uint_as_float(static_cast<uint32_t>(p.vc[at + i]) << 16);
    }
    for (int i = 0; i < per; ++i) p.out[seq * p.os + h * p.D + per * lane + i] = f2bf_bits(n ? acc[i] / sum : 0.f);
    if (p.lse && lane == 0) p.lse[w] = n ? top + logf(sum) : -INFINITY;
}

}  // namespace attn
}  // namespace kda
