// kda_gdn_step.cuh -- the gated delta rule with one decay per head, token by token: single tokens against a state kept
// in place, and short prompts.
//   a = -exp(A_log[h]) softplus(a_t + dt_bias[h]),  b = sigmoid(beta_t)
//   S <- e^a S (I - b k k^T) + b v k^T,  out = scale S q            (S: 128 x 128 per value head, stored [v][k])
// A row s of S changes by n k with n = b (v - e^a s.k), and its output is e^a s.q + n k.q, so both of its dot products
// are taken from the old row, together. A warp owns ROWS rows, four of the 128 key channels per lane, in fp32 registers
// from the first token to the last; the 2 ROWS sums go through a reduce-scatter butterfly (sixteen exchanges for eight
// rows), after which the rows' n are handed back to all lanes.
// Bound by the state's bytes for single tokens: 128 sequences of 16 heads, 268 MB of fp32 state read and written, take
// 40.5 us on the device, 6.6 TB/s, what a copy reaches. Over more tokens the sums bound it, 0.35 us a token and more.
#pragma once
#include "blk_common.cuh"

namespace kda {
namespace gdn {

constexpr int ROWS = 8;        // state rows per warp
constexpr int STEP_THREADS = 128;
constexpr float L2_EPS = 1e-6f;
// Sequences of up to this many tokens go token by token: sooner done than by chunks at every size, and more exact. us for
// 8 tokens: 6.7 against 12.6 (1 sequence of 8 heads), 10.6 against 13.9 (8 of 16), 59 against 93 (64 of 16); for 12: 14.3
// against 13.8 (8 of 16); for 16: 11.4 against 12.9, and 105 against 93 (64 of 16).
constexpr int STEP_TOKENS = 8;

struct GdnParams {
    const uint16_t *q, *k, *v, *a, *beta;
    uint16_t *out;
    long long qs, ks, vs, as, bs, os;   // elements between tokens
    const float *A_log, *dt_bias;
    const void *init;
    void *fin;
    const int64_t *cu;
    int init_dtype, fin_dtype;
    int T, H, HK, nseq, total;
    float scale;
    int l2;                             // queries and keys are normalised here
    int split;                          // a packed call of two launches: short sequences token by token, the others by chunks
};

__device__ __forceinline__ float softplus(float u) { return u > 20.f ? u : log1pf(expf(u)); }
__device__ __forceinline__ float sigmoid(float u) { return 1.f / (1.f + expf(-u)); }

__device__ __forceinline__ Span gdn_span(const GdnParams &p, int seq)
{
    if (p.cu) {
        const long long b = p.cu[seq], e = p.cu[seq + 1];
        if (b < 0 || e < b || e > p.total) return {0, 0, false};
        return {static_cast<int>(b), static_cast<int>(e - b), true};
    }
    return {seq * p.T, p.T, true};
}

__device__ __forceinline__ size_t state_elems(const GdnParams &p) { return static_cast<size_t>(p.nseq) * p.H * DH * DH; }

// Rows r0 .. r0 + 7 of one (sequence, head) through the sequence's tokens: every lane of a warp together.
__device__ __forceinline__ void walk_rows(const GdnParams &p, int seq, int h, const Span &sp, int r0)
{
    const int lane = threadIdx.x & 31;
    const size_t st = ((static_cast<size_t>(seq) * p.H + h) * DH + r0) * DH + 4 * lane;
    float2 s[ROWS][2];  // paired arithmetic
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        s[r][0] = s[r][1] = make_float2(0.f, 0.f);
        if (p.init && gmem_ok(st + r * DH, 4, state_elems(p))) {
            if (p.init_dtype == KDA_DTYPE_FP32) {
                const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.init) + st + r * DH);
                s[r][0] = make_float2(v.x, v.y);
                s[r][1] = make_float2(v.z, v.w);
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.init) + st + r * DH);
                s[r][0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
                s[r][1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
            }
        }
    }
    const float A2 = -expf(__ldg(p.A_log + h)) * LOG2E, bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f;
    const long long bos = sp.bos, hk = h / (p.H / p.HK);
    const uint16_t *qp = p.q + bos * p.qs + hk * DH + 4 * lane, *kp = p.k + bos * p.ks + hk * DH + 4 * lane;
    const uint16_t *vp = p.v + bos * p.vs + static_cast<long long>(h) * DH + r0;
    const uint16_t *ap = p.a + bos * p.as + h, *bp = p.beta + bos * p.bs + h;
    uint16_t *op = p.out + bos * p.os + static_cast<long long>(h) * DH + r0 + ((lane >> 1) & 7);
    uint4 vn = make_uint4(0u, 0u, 0u, 0u);
    uint2 qn = make_uint2(0u, 0u), kn = qn;
    float keeps = 0.f, steps = 0.f;  // of token 32 i + lane
    uint32_t an = 0u, bn = 0u;
    auto fetch = [&](int t) {  // token t's inputs, one token ahead of their use
        vn = *reinterpret_cast<const uint4 *>(vp + t * p.vs);
        qn = *reinterpret_cast<const uint2 *>(qp + t * p.qs);
        kn = *reinterpret_cast<const uint2 *>(kp + t * p.ks);
    };
    auto fetch_gate = [&](int t) {  // of 32 tokens, a lane each
        if (t + lane < sp.len) {
            an = ap[(t + lane) * p.as];
            bn = bp[(t + lane) * p.bs];
        }
    };
    fetch_gate(0);
    if (sp.len > 0) fetch(0);
    for (int t = 0; t < sp.len; ++t) {
        float2 k[2] = {make_float2(bf16_lo(kn.x), bf16_hi(kn.x)), make_float2(bf16_lo(kn.y), bf16_hi(kn.y))};
        float2 q[2] = {make_float2(bf16_lo(qn.x), bf16_hi(qn.x)), make_float2(bf16_lo(qn.y), bf16_hi(qn.y))};
        // v of row (lane >> 1) & 7, whose n this lane works out
        const uint32_t vw = lane & 8 ? (lane & 4 ? vn.w : vn.z) : (lane & 4 ? vn.y : vn.x);
        const float v = lane & 2 ? bf16_hi(vw) : bf16_lo(vw);
        if (t + 1 < sp.len) fetch(t + 1);
        if ((t & 31) == 0) {
            keeps = exp2f(A2 * softplus(__uint_as_float(an << 16) + bias));
            steps = sigmoid(__uint_as_float(bn << 16));
            fetch_gate(t + 32);
        }
        const float keep = __shfl_sync(0xffffffffu, keeps, t & 31), b = __shfl_sync(0xffffffffu, steps, t & 31);
        auto dot = [](const float2(&x)[2], const float2(&y)[2]) {
            const float2 u = ffma2(x[0], y[0], fmul2(x[1], y[1]));
            return u.x + u.y;
        };
        float kq = dot(k, q);
        float fq = p.scale;
        if (p.l2) {
            float kk = dot(k, k), qq = dot(q, q);
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) {
                kk += __shfl_xor_sync(0xffffffffu, kk, m);
                qq += __shfl_xor_sync(0xffffffffu, qq, m);
            }
            const float fk = 1.f / sqrtf(kk + L2_EPS);
            k[0] = fmul2(k[0], make_float2(fk, fk));
            k[1] = fmul2(k[1], make_float2(fk, fk));
            fq *= 1.f / sqrtf(qq + L2_EPS);
            kq *= fk;
        }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, m);
        float y[2 * ROWS];  // s.q of the rows, then s.k
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            y[r] = dot(s[r], q);
            y[ROWS + r] = dot(s[r], k);
        }
        // reduce-scatter: lane l ends with sum l >> 1
#pragma unroll
        for (int m = 16, n = ROWS; m >= 2; m >>= 1, n >>= 1) {
            const bool up = lane & m;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float mine = up ? y[i + n] : y[i], send = up ? y[i] : y[i + n];
                y[i] = mine + __shfl_xor_sync(0xffffffffu, send, m);
            }
        }
        y[0] += __shfl_xor_sync(0xffffffffu, y[0], 1);
        const float n = b * (v - keep * y[0]);  // of use in lanes 16 and up, which hold s.k
        const float n_row = __shfl_sync(0xffffffffu, n, lane | 16);
        if (lane < 16 && (lane & 1) == 0) op[t * p.os] = f2bf_bits(fq * fmaf(n_row, kq, keep * y[0]));
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const float nr = __shfl_sync(0xffffffffu, n, 16 + 2 * r);
#pragma unroll
            for (int j = 0; j < 2; ++j) s[r][j] = ffma2(make_float2(keep, keep), s[r][j], fmul2(make_float2(nr, nr), k[j]));
        }
    }
    if (!p.fin) return;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        if (gmem_ok(st + r * DH, 4, state_elems(p))) {
            if (p.fin_dtype == KDA_DTYPE_FP32)
                *reinterpret_cast<float4 *>(static_cast<float *>(p.fin) + st + r * DH) = make_float4(s[r][0].x, s[r][0].y, s[r][1].x, s[r][1].y);
            else
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.fin) + st + r * DH) =
                    make_uint2(pack_bf16(s[r][0].x, s[r][0].y), pack_bf16(s[r][1].x, s[r][1].y));
        }
}

__global__ void __launch_bounds__(STEP_THREADS) kda_gdn_step_kernel(const GdnParams p, long long nwarps)
{
    const long long w = static_cast<long long>(blockIdx.x) * (STEP_THREADS / 32) + (threadIdx.x >> 5);
    if (p.cu && blockIdx.x == 0) blk::check_bounds(p.cu, p.nseq, p.total);
    if (w >= nwarps) return;
    constexpr int RB = DH / ROWS;                    // row blocks per head
    const long long unit = w / RB;                   // (sequence, head)
    const int h = static_cast<int>(unit % p.H), seq = static_cast<int>(unit / p.H);
    const Span sp = gdn_span(p, seq);
    if (!sp.ok || (p.split && sp.len > STEP_TOKENS)) return;  // not ok: flagged by check_bounds
    walk_rows(p, seq, h, sp, static_cast<int>(w % RB) * ROWS);
}

}  // namespace gdn
}  // namespace kda
