// kda_ssm_step.cuh -- the selective state-space recurrence token by token: single tokens against a
// state kept in place, and short prompts.
//   delta = softplus(dt + dt_bias[h]),  a = -exp(A_log[h]) delta
//   S <- exp(a) S + delta x b^T,  out = S c + D[h] x          (S: P x 128 per head)
// A warp owns ROWS rows of one head's state, four of the 128 state channels per lane (16 bytes of
// fp32 state per row and lane), in fp32 registers from the first token to the last; the row sums
// S c go through a reduce-scatter butterfly (nine exchanges for eight rows). One token reads and
// writes the state once, so the step is bound by HBM (128 sequences x 16 heads of 128, fp32 states: 43.4 us,
// 6.2 TB/s, 93 % of a plain copy); a prompt walks its tokens one after another and is bound by the latency
// of one token's chain.
// A few tokens against many states are bound by issue and the chain: 1024 sequences of 8 tokens, 16 heads of 128, take
// 552 us (658 with scalar arithmetic and every lane working out each token's step size and decay, which a lane now
// does for one token of 32).
#pragma once
#include "blk_common.cuh"

namespace kda {
namespace ssm {

constexpr int NS = 128;        // state channels
constexpr int ROWS = 8;        // state rows per warp
constexpr int STEP_THREADS = 128;
// The log2 decay of one token is held at or above this: 2^-160 is zero in fp32 either way, and a running sum over 32
// tokens stays above -5120, so that each of its at most seven roundings is below 2^-12. The difference of two such sums is
// off by 2^-8 at worst, and only behind tokens whose decay is at the limit; where the sums stay above -64, by 2^-15.
constexpr float MIN_LOG2_DECAY = -160.f;

struct SsmParams {
    const uint16_t *x, *dt, *b, *c;
    uint16_t *out;
    long long xs, dts, bs, cs, os;   // elements between tokens
    const float *A_log, *D, *dt_bias;
    const void *init;
    void *fin;
    const int64_t *cu;
    int init_dtype, fin_dtype;
    int T, H, P, G, nseq, total;
};

__device__ __forceinline__ float softplus(float u) { return u > 20.f ? u : log1pf(expf(u)); }

__device__ __forceinline__ Span ssm_span(const SsmParams &p, int seq)
{
    if (p.cu) {
        const long long b = p.cu[seq], e = p.cu[seq + 1];
        if (b < 0 || e < b || e > p.total) return {0, 0, false};
        return {static_cast<int>(b), static_cast<int>(e - b), true};
    }
    return {seq * p.T, p.T, true};
}

__global__ void __launch_bounds__(STEP_THREADS) kda_ssm_step_kernel(const SsmParams p, long long nwarps)
{
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * (STEP_THREADS / 32) + (threadIdx.x >> 5);
    if (p.cu && blockIdx.x == 0) blk::check_bounds(p.cu, p.nseq, p.total);
    if (w >= nwarps) return;
    const int rb = p.P / ROWS;                       // row blocks per head
    const long long unit = w / rb;                   // (sequence, head)
    const int r0 = static_cast<int>(w % rb) * ROWS;
    const int h = static_cast<int>(unit % p.H), seq = static_cast<int>(unit / p.H);
    const int g = h / (p.H / p.G);
    const Span sp = ssm_span(p, seq);
    if (!sp.ok) return;  // flagged by check_bounds
    const size_t st = (static_cast<size_t>(unit) * p.P + r0) * NS + 4 * lane;
    const size_t st_elems = static_cast<size_t>(p.nseq) * p.H * p.P * NS;
    float2 s[ROWS][2];  // paired arithmetic
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        s[r][0] = s[r][1] = make_float2(0.f, 0.f);
        if (p.init && gmem_ok(st + r * NS, 4, st_elems)) {
            if (p.init_dtype == KDA_DTYPE_FP32) {
                const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.init) + st + r * NS);
                s[r][0] = make_float2(v.x, v.y);
                s[r][1] = make_float2(v.z, v.w);
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.init) + st + r * NS);
                s[r][0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
                s[r][1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
            }
        }
    }
    const float A2 = -expf(__ldg(p.A_log + h)) * LOG2E;
    const float bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f, Dh = p.D ? __ldg(p.D + h) : 0.f;
    const uint16_t *xp = p.x + static_cast<long long>(sp.bos) * p.xs + static_cast<long long>(h) * p.P + r0;
    const uint16_t *dp = p.dt + static_cast<long long>(sp.bos) * p.dts + h;
    const uint16_t *bp = p.b + static_cast<long long>(sp.bos) * p.bs + static_cast<long long>(g) * NS + 4 * lane;
    const uint16_t *cp = p.c + static_cast<long long>(sp.bos) * p.cs + static_cast<long long>(g) * NS + 4 * lane;
    uint16_t *op = p.out + static_cast<long long>(sp.bos) * p.os + static_cast<long long>(h) * p.P + r0 + (lane >> 2);
    uint4 xn = make_uint4(0u, 0u, 0u, 0u);
    uint2 bn = make_uint2(0u, 0u), cn = bn;
    float deltas = 0.f, keeps = 0.f;  // of token 32 k + lane
    auto fetch = [&](int t) {  // token t's inputs, one token ahead of their use
        xn = *reinterpret_cast<const uint4 *>(xp + t * p.xs);
        bn = *reinterpret_cast<const uint2 *>(bp + t * p.bs);
        cn = *reinterpret_cast<const uint2 *>(cp + t * p.cs);
    };
    // dt of 32 tokens, a lane each
    auto fetch_dt = [&](int t) { return t + lane < sp.len ? static_cast<uint32_t>(dp[(t + lane) * p.dts]) : 0u; };
    uint32_t dn = fetch_dt(0);
    if (sp.len > 0) fetch(0);
    for (int t = 0; t < sp.len; ++t) {
        float x[8];
        blk::unpack8(xn, x);
        const float2 bf[2] = {make_float2(bf16_lo(bn.x), bf16_hi(bn.x)), make_float2(bf16_lo(bn.y), bf16_hi(bn.y))};
        const float2 cf[2] = {make_float2(bf16_lo(cn.x), bf16_hi(cn.x)), make_float2(bf16_lo(cn.y), bf16_hi(cn.y))};
        // x of row lane >> 2, whose output this lane may write
        const uint32_t xw = lane & 16 ? (lane & 8 ? xn.w : xn.z) : (lane & 8 ? xn.y : xn.x);
        const float xo = lane & 4 ? bf16_hi(xw) : bf16_lo(xw);
        if (t + 1 < sp.len) fetch(t + 1);
        if ((t & 31) == 0) {
            deltas = softplus(__uint_as_float(dn << 16) + bias);
            keeps = exp2f(A2 * deltas);
            dn = fetch_dt(t + 32);
        }
        const float delta = __shfl_sync(0xffffffffu, deltas, t & 31), keep = __shfl_sync(0xffffffffu, keeps, t & 31);
        float y[8];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const float dx = delta * x[r];
#pragma unroll
            for (int j = 0; j < 2; ++j) s[r][j] = ffma2(make_float2(keep, keep), s[r][j], fmul2(make_float2(dx, dx), bf[j]));
            const float2 u = ffma2(s[r][0], cf[0], fmul2(s[r][1], cf[1]));
            y[r] = u.x + u.y;
        }
        // reduce-scatter: lane l ends with the sum of row l >> 2
#pragma unroll
        for (int m = 16, n = 4; m >= 4; m >>= 1, n >>= 1) {
            const bool up = lane & m;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float keepv = up ? y[i + n] : y[i], send = up ? y[i] : y[i + n];
                y[i] = keepv + __shfl_xor_sync(0xffffffffu, send, m);
            }
        }
        y[0] += __shfl_xor_sync(0xffffffffu, y[0], 2);
        y[0] += __shfl_xor_sync(0xffffffffu, y[0], 1);
        if ((lane & 3) == 0) op[t * p.os] = f2bf_bits(p.D ? fmaf(Dh, xo, y[0]) : y[0]);
    }
    if (!p.fin) return;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        if (gmem_ok(st + r * NS, 4, st_elems)) {
            if (p.fin_dtype == KDA_DTYPE_FP32)
                *reinterpret_cast<float4 *>(static_cast<float *>(p.fin) + st + r * NS) = make_float4(s[r][0].x, s[r][0].y, s[r][1].x, s[r][1].y);
            else
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.fin) + st + r * NS) =
                    make_uint2(pack_bf16(s[r][0].x, s[r][0].y), pack_bf16(s[r][1].x, s[r][1].y));
        }
}

}  // namespace ssm
}  // namespace kda
