// kda_rope.cuh -- heads of queries and keys normed and turned by their position, and keys and values on their way into
// a paged cache.
//   n = x rsqrt(mean x^2 + eps) w                     (or n = x)
//   (n_i, n_j) -> (n_i cos - n_j sin, n_j cos + n_i sin),   angle = position inv_freq[pair]
// where pair i is channels (i, i + R/2), or (2 i, 2 i + 1); channels from R on are not turned.
// Angles: a float holds a far position's angle to no better than 2^-24 of it, which at position 100,000 is a hundredth of
// a radian. The turn is therefore counted in whole turns, as a 64-bit fixed-point fraction: inv_freq / (2 pi) is an
// integer F of 2^-64 turns, position F wraps as turns do, and its upper 32 bits, rounded, are the angle. F is off by less than
// 1 + inv_freq / 256 units (2 / pi has 64 bits, and F is cut off), so an angle is off by less than 2^-33 + |position| (1 +
// inv_freq / 256) 2^-64 turns: 2^-31 below position 2^32 for frequencies up to 64. It is taken from the nearest quarter turn
// before it becomes a float, whose 24 bits then hold it to 2^-28 turns at most and the smaller of cosine and sine to 2^-24 of
// itself; no 64-bit floating point is needed.
// Bound by HBM where there are many tokens: 32,768 of 20 heads of 128 take 63.5 us, 5.3 TB/s; 65,519 packed ones appended
// with 8 key heads of 128, .54 GB, 92 us, 5.8 TB/s. For single tokens the launch and one chain of loads are all: 6 us.
#pragma once
#include "blk_common.cuh"

namespace kda {
namespace rope {

constexpr int THREADS = 128;
constexpr int MAX_D = 256;
constexpr int MAX_TOKENS = 16; // of a CTA
constexpr int BLOCK = 4;       // tokens that a warp takes through a group of heads

struct Turn {
    const int64_t *positions;  // per token
    const float *inv_freq;     // [R / 2]
    int R;                     // channels that are turned, a multiple of 16
    int inter;                 // pairs are neighbours
};

struct HeadNorm {
    int norm;
    float eps;
};

// inv_freq / (2 pi) in units of 2^-64 turns, modulo one turn. f = m 2^e with an integer m below 2^24, and 2 / pi in 64
// bits is 2^66 / (2 pi), so that F = m (2 / pi) 2^(e - 2).
__device__ __forceinline__ uint64_t turns_per_step(float f)
{
    const uint32_t bits = __float_as_uint(f), ex = (bits >> 23) & 255u;
    const uint64_t m = ex ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const int s = 2 - (static_cast<int>(ex ? ex : 1u) - 150);  // right shift of the 88-bit product
    constexpr uint64_t C = 0xA2F9836E4E44152AULL;               // 2 / pi, rounded to 64 bits
    const uint64_t lo = m * C, hi = __umul64hi(m, C);
    uint64_t F = 0;
    if (s >= 128)
        F = 0;
    else if (s >= 64)
        F = hi >> (s - 64);
    else if (s > 0)
        F = (hi << (64 - s)) | (lo >> s);
    else if (s > -64)
        F = lo << -s;
    return bits >> 31 ? 0 - F : F;
}

// cosine and sine of the angle at `position`
__device__ __forceinline__ float2 turn_at(int64_t position, uint64_t F)
{
    const uint32_t a = static_cast<uint32_t>((static_cast<uint64_t>(position) * F + 0x80000000u) >> 32);  // 2^-32 turns
    const uint32_t n = (a + 0x20000000u) >> 30;                                                           // the nearest quarter
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(a - (n << 30))) * 0x1p-31f, &s, &c);
    const float x = n & 1 ? -s : c, y = n & 1 ? c : s;
    return n & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

// A head is held by D / 16 neighbouring lanes, two vectors of eight channels each, of the part that is turned both members
// of eight pairs. First and second vectors of neighbouring lanes are neighbours, so that an access covers whole sectors
// (32,768 tokens of 20 heads of 128, 32 channels turned: 78 us with a lane's vectors side by side, 63 so).
template <int D, bool INTER>
struct Lane {
    static constexpr int LANES = D / 16, HEADS = 32 / LANES;  // of a head, and heads of a warp
    int v0, v1;    // first channel of either vector
    int q0, q1;    // where either's turns begin in the table (interleaved pairs; else q0 is both's)
    bool t0, t1;   // turned
    __device__ __forceinline__ explicit Lane(int R)
    {
        const int j = threadIdx.x % LANES, half = R / 16;  // vectors in half of the turned part
        if (INTER) {
            v0 = 8 * j;
            v1 = 8 * (j + LANES);
            q0 = j;
            q1 = j + LANES;
            t0 = v0 < R;
            t1 = v1 < R;
        } else {
            const bool in = j < half;
            v0 = in ? 8 * j : 8 * (j + half);
            v1 = in ? 8 * (j + half) : 8 * (j + LANES);
            q0 = q1 = j;
            t0 = t1 = in;
        }
    }
};

// The CTA's turns: per token R / 4 quadruples (cos, cos, sin, sin) of two pairs. A lane reads those of its eight pairs (four,
// of a vector of interleaved ones) in steps, and the quadruples of neighbouring lanes' steps lie next to each other.
template <bool INTER>
__device__ __forceinline__ void make_table(float *table, const Turn &t, long long tok0, int tokens)
{
    constexpr int G = INTER ? 4 : 8;  // pairs of a lane's read
    const int half = t.R / 2;
    for (int i = threadIdx.x; i < half * tokens; i += blockDim.x) {
        const int tk = i / half, f = i - tk * half;
        const float2 cs = turn_at(__ldg(t.positions + tok0 + tk), turns_per_step(__ldg(t.inv_freq + f)));
        float *at = table + 4 * (tk * (half / 2) + ((f % G) >> 1) * (half / G) + f / G) + (f & 1);
        at[0] = cs.x;
        at[2] = cs.y;
    }
}

__device__ __forceinline__ void load_weights(const float *w, int c, float2 (&f)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(1.f, 1.f);
    if (w) blk::load8f(w + c, f);
}

// Norm and turn of one head; wa, wb: the lane's weights; table: the token's turns.
template <int D, bool INTER>
__device__ __forceinline__ void norm_and_turn(float2 (&a)[4], float2 (&b)[4], bool norm, float eps, const float2 (&wa)[4], const float2 (&wb)[4],
                                              const Lane<D, INTER> &l, const float4 *table, int half)
{
    if (norm) {
        float2 ss = fmul2(a[0], a[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) ss = ffma2(a[i], a[i], ss);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = ffma2(b[i], b[i], ss);
        float sum = ss.x + ss.y;
#pragma unroll
        for (int m = D / 32; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const float f = rsqrtf(fmaf(sum, 1.f / D, eps));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = fmul2(a[i], fmul2(wa[i], make_float2(f, f)));
            b[i] = fmul2(b[i], fmul2(wb[i], make_float2(f, f)));
        }
    }
    if (INTER) {  // pairs inside the vectors
        auto turn = [&](float2(&x)[4], int q) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 t = table[i * (half / 4) + q];
                x[2 * i] = make_float2(x[2 * i].x * t.x - x[2 * i].y * t.z, x[2 * i].y * t.x + x[2 * i].x * t.z);
                x[2 * i + 1] = make_float2(x[2 * i + 1].x * t.y - x[2 * i + 1].y * t.w, x[2 * i + 1].y * t.y + x[2 * i + 1].x * t.w);
            }
        };
        if (l.t0) turn(a, l.q0);
        if (l.t1) turn(b, l.q1);
    } else if (l.t0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 t = table[i * (half / 8) + l.q0];
            const float2 c = make_float2(t.x, t.y), s = make_float2(t.z, t.w), x = a[i], y = b[i];
            a[i] = fsub2(fmul2(x, c), fmul2(y, s));
            b[i] = ffma2(x, s, fmul2(y, c));
        }
    }
}

struct QkParams {
    const uint16_t *q, *k;
    uint16_t *qo, *ko;
    long long qs, ks, qos, kos;  // elements between tokens
    const float *qw, *kw;
    Turn turn;
    HeadNorm hn;
    long long M;
    int H, HK, tokens;           // tokens: of one CTA
};

// A CTA makes the turns of its tokens, and its warps take blocks of four tokens through groups of heads: four tokens' loads
// are in flight, and what belongs to a head (addresses, weights) is worked out once for them.
template <int D, bool INTER>
__global__ void __launch_bounds__(THREADS) kda_qk_rope_kernel(const QkParams p)
{
    extern __shared__ __align__(16) float table[];
    using L = Lane<D, INTER>;
    const long long tok0 = static_cast<long long>(blockIdx.x) * p.tokens;
    const int n = static_cast<int>(min(static_cast<long long>(p.tokens), p.M - tok0)), half = p.turn.R / 2;
    const int warp = threadIdx.x >> 5, mine = (threadIdx.x & 31) / L::LANES, heads = p.H + p.HK;
    const int groups = (heads + L::HEADS - 1) / L::HEADS, units = groups * ((n + BLOCK - 1) / BLOCK);
    const L l(p.turn.R);
    uint4 x[BLOCK][2];
    long long at = 0, stride = 0;
    int hd = 0, t0 = 0;
    auto fetch = [&](int u) {  // unit u: a group of heads, four tokens
        t0 = u / groups * BLOCK;
        hd = u % groups * L::HEADS + mine;
        const bool is_q = hd < p.H;
        stride = is_q ? p.qs : p.ks;
        at = (tok0 + t0) * stride + (is_q ? hd : hd - p.H) * D;
        const uint16_t *src = is_q ? p.q : p.k;
        const long long end = (p.M - 1) * stride + (is_q ? p.H : p.HK) * D;
#pragma unroll
        for (int b = 0; b < BLOCK; ++b) {
            x[b][0] = x[b][1] = make_uint4(0u, 0u, 0u, 0u);
            if (hd < heads && t0 + b < n && gmem_ok(at + b * stride, D, end)) {
                x[b][0] = *reinterpret_cast<const uint4 *>(src + at + b * stride + l.v0);
                x[b][1] = *reinterpret_cast<const uint4 *>(src + at + b * stride + l.v1);
            }
        }
    };
    if (warp < units) fetch(warp);  // ahead of the table, whose chain is long
    make_table<INTER>(table, p.turn, tok0, n);
    __syncthreads();
    for (int u = warp; u < units; u += THREADS / 32) {
        if (u != warp) fetch(u);
        const bool is_q = hd < p.H;
        float2 wa[4], wb[4];
        load_weights(is_q ? p.qw : p.kw, l.v0, wa);
        load_weights(is_q ? p.qw : p.kw, l.v1, wb);
        uint16_t *dst = is_q ? p.qo : p.ko;
        const long long ostride = is_q ? p.qos : p.kos, end = (p.M - 1) * ostride + (is_q ? p.H : p.HK) * D;
        const long long to = (tok0 + t0) * ostride + (is_q ? hd : hd - p.H) * D;
#pragma unroll
        for (int b = 0; b < BLOCK; ++b) {
            if (t0 + b >= n) break;  // the same for the whole warp
            float2 f[4], g[4];
            blk::unpack8(x[b][0], f);
            blk::unpack8(x[b][1], g);
            norm_and_turn<D, INTER>(f, g, p.hn.norm, p.hn.eps, wa, wb, l, reinterpret_cast<const float4 *>(table) + (t0 + b) * (half / 2), half);
            if (hd < heads && gmem_ok(to + b * ostride, D, end)) {
                *reinterpret_cast<uint4 *>(dst + to + b * ostride + l.v0) = blk::pack8(f);
                *reinterpret_cast<uint4 *>(dst + to + b * ostride + l.v1) = blk::pack8(g);
            }
        }
    }
}

// ------------------------------------------------------------------------------------------ a paged cache

// Pages of [heads, page_size, D] elements, page_stride elements apart; page_size a power of two.
struct Pages {
    long long stride;
    const int32_t *table;  // [sequences, width]
    int width, count, shift;
};

struct AppendParams {
    const uint16_t *k, *v;
    uint16_t *kc, *vc;
    long long ks, vs;
    const float *kw;
    Turn turn;
    HeadNorm hn;
    Pages pages;
    const int64_t *cu;
    long long M;
    int T, nseq, HK, tokens;
};

// Where a token's rows stand in the cache (of head 0), or -1 where it has none: positions below zero are padding.
__device__ __forceinline__ long long slot_of(const AppendParams &p, long long tok, int D)
{
    const int64_t pos = __ldg(p.turn.positions + tok);
    if (pos < 0) return -1;
    long long seq = tok / p.T;
    if (p.cu) {
        const blk::Enclosing e = blk::find_sequence(p.cu, p.nseq, p.M, tok);
        if (!e.ok) return -1;  // flagged by check_bounds
        seq = e.seq;
    }
    const int64_t at = pos >> p.pages.shift;
    int page = -1;
    if (at < p.pages.width) page = __ldg(p.pages.table + seq * p.pages.width + at);
    if (page < 0 || page >= p.pages.count) {
        atomicOr(&g_dev_error, DEVERR_PAGES);
        return -1;
    }
    return page * p.pages.stride + (pos & ((1 << p.pages.shift) - 1)) * D;
}

template <int D, bool INTER>
__global__ void __launch_bounds__(THREADS) kda_kv_append_kernel(const AppendParams p)
{
    extern __shared__ __align__(16) float table[];
    __shared__ long long slots[MAX_TOKENS];
    using L = Lane<D, INTER>;
    constexpr int B = BLOCK / 2;  // tokens of a block: keys and values
    const long long tok0 = static_cast<long long>(blockIdx.x) * p.tokens;
    const int n = static_cast<int>(min(static_cast<long long>(p.tokens), p.M - tok0)), half = p.turn.R / 2;
    if (p.cu && blockIdx.x == 0) blk::check_bounds(p.cu, p.nseq, p.M);
    const int warp = threadIdx.x >> 5, mine = (threadIdx.x & 31) / L::LANES;
    const int groups = (p.HK + L::HEADS - 1) / L::HEADS, units = groups * ((n + B - 1) / B);
    const L l(p.turn.R);
    const long long page_size = 1LL << p.pages.shift, cache = (p.pages.count - 1) * p.pages.stride + p.HK * page_size * D;
    uint4 x[B][2], y[B][2];
    int hd = 0, t0 = 0;
    auto fetch = [&](int u) {
        t0 = u / groups * B;
        hd = u % groups * L::HEADS + mine;
        const long long at = (tok0 + t0) * p.ks + hd * D, vat = (tok0 + t0) * p.vs + hd * D;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            x[b][0] = x[b][1] = y[b][0] = y[b][1] = make_uint4(0u, 0u, 0u, 0u);
            if (hd < p.HK && t0 + b < n && gmem_ok(at + b * p.ks, D, (p.M - 1) * p.ks + p.HK * D) && gmem_ok(vat + b * p.vs, D, (p.M - 1) * p.vs + p.HK * D)) {
                x[b][0] = *reinterpret_cast<const uint4 *>(p.k + at + b * p.ks + l.v0);
                x[b][1] = *reinterpret_cast<const uint4 *>(p.k + at + b * p.ks + l.v1);
                y[b][0] = *reinterpret_cast<const uint4 *>(p.v + vat + b * p.vs + l.v0);
                y[b][1] = *reinterpret_cast<const uint4 *>(p.v + vat + b * p.vs + l.v1);
            }
        }
    };
    if (warp < units) fetch(warp);  // ahead of the table and the look-up of pages, whose chains are long
    if (threadIdx.x < n) slots[threadIdx.x] = slot_of(p, tok0 + threadIdx.x, D);
    make_table<INTER>(table, p.turn, tok0, n);
    float2 wa[4], wb[4];
    load_weights(p.kw, l.v0, wa);
    load_weights(p.kw, l.v1, wb);
    __syncthreads();
    for (int u = warp; u < units; u += THREADS / 32) {
        if (u != warp) fetch(u);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (t0 + b >= n) break;  // the same for the whole warp
            float2 f[4], g[4];
            blk::unpack8(x[b][0], f);
            blk::unpack8(x[b][1], g);
            norm_and_turn<D, INTER>(f, g, p.hn.norm, p.hn.eps, wa, wb, l, reinterpret_cast<const float4 *>(table) + (t0 + b) * (half / 2), half);
            const long long slot = slots[t0 + b], dst = slot + hd * page_size * D;
            if (slot >= 0 && hd < p.HK && gmem_ok(dst, D, cache)) {
                *reinterpret_cast<uint4 *>(p.kc + dst + l.v0) = blk::pack8(f);
                *reinterpret_cast<uint4 *>(p.kc + dst + l.v1) = blk::pack8(g);
                *reinterpret_cast<uint4 *>(p.vc + dst + l.v0) = y[b][0];
                *reinterpret_cast<uint4 *>(p.vc + dst + l.v1) = y[b][1];
            }
        }
    }
}

}  // namespace rope
}  // namespace kda
