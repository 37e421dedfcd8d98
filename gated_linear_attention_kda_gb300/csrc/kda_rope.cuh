// kda_rope.cuh -- heads of queries and keys normed and turned by their position, and keys and values on their way into
// a paged cache.
//   n = x rsqrt(mean x^2 + eps) w                     (or n = x)
//   (n_i, n_j) -> (n_i cos - n_j sin, n_j cos + n_i sin),   angle = position inv_freq[pair]
// where pair i is channels (i, i + R/2), or (2 i, 2 i + 1); channels from R on are not turned.
// Angles: a float holds a far position's angle to no better than 2^-24 of it, which at position 100,000 is a hundredth of
// a radian. The turn is therefore counted in whole turns, as a 64-bit fixed-point fraction: inv_freq / (2 pi) is an
// integer F of 2^-64 turns, position F wraps as turns do, and its upper 32 bits are the angle. F is off by at most one
// unit, so a position below 2^31 is off by less than 2^-33 turns; no 64-bit floating point is needed.
#pragma once
#include "blk_common.cuh"

namespace kda {
namespace rope {

constexpr int THREADS = 128;
constexpr int MAX_D = 256;

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
    const int32_t a = static_cast<int32_t>((static_cast<uint64_t>(position) * F) >> 32);  // 2^-32 turns, in [-1/2, 1/2)
    float s, c;
    sincospif(static_cast<float>(a) * 0x1p-31f, &s, &c);
    return make_float2(c, s);
}

// A lane owns two vectors of eight channels of a head: of the part that is turned, both members of eight pairs.
struct Vectors {
    int v0, v1;    // first channel of either
    bool turned;
};
__device__ __forceinline__ Vectors vectors_of(int j, int R, bool inter)
{
    const int half = R / 16;  // vectors in half of the turned part
    if (inter) return {16 * j, 16 * j + 8, j < half};
    if (j < half) return {8 * j, 8 * (j + half), true};
    return {16 * j, 16 * j + 8, false};
}

// Norm and turn of one head held by `lanes` neighbouring lanes; w: the lane's 16 weights; cs: table of the token.
template <bool INTER>
__device__ __forceinline__ void norm_and_turn(float (&a)[8], float (&b)[8], bool norm, float eps, float inv_d, int lanes, const float (&w)[16],
                                              bool turned, const float2 *cs)
{
    if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
        for (int m = lanes >> 1; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float f = rsqrtf(fmaf(ss, inv_d, eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] *= f * w[i];
            b[i] *= f * w[8 + i];
        }
    }
    if (!turned) return;
    if (INTER) {  // pairs inside the vectors
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 t0 = cs[i / 2], t1 = cs[4 + i / 2];
            const float x = a[i], y = b[i];
            a[i] = x * t0.x - a[i + 1] * t0.y;
            a[i + 1] = a[i + 1] * t0.x + x * t0.y;
            b[i] = y * t1.x - b[i + 1] * t1.y;
            b[i + 1] = b[i + 1] * t1.x + y * t1.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 t = cs[i];
            const float x = a[i];
            a[i] = x * t.x - b[i] * t.y;
            b[i] = b[i] * t.x + x * t.y;
        }
    }
}

// The CTA's table of cosines and sines: `tokens` rows of R / 2 pairs.
__device__ __forceinline__ void make_table(float2 *table, const Turn &t, long long tok0, int tokens)
{
    const int half = t.R / 2;
    for (int i = threadIdx.x; i < half * tokens; i += blockDim.x) {
        const int tk = i / half, f = i - tk * half;
        table[i] = turn_at(__ldg(t.positions + tok0 + tk), turns_per_step(__ldg(t.inv_freq + f)));
    }
}

__device__ __forceinline__ void load_weights(const float *w, const Vectors &v, float (&f)[16])
{
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = b[i] = 1.f;
    if (w) {
        blk::load8f(w + v.v0, a);
        blk::load8f(w + v.v1, b);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = a[i];
        f[8 + i] = b[i];
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
    int H, HK, D, tokens;        // tokens: of one CTA
};

template <bool INTER>
__global__ void __launch_bounds__(THREADS) kda_qk_rope_kernel(const QkParams p)
{
    extern __shared__ float2 table[];
    const long long tok0 = static_cast<long long>(blockIdx.x) * p.tokens;
    const int n = static_cast<int>(min(static_cast<long long>(p.tokens), p.M - tok0));
    make_table(table, p.turn, tok0, n);
    __syncthreads();
    const int lanes = p.D / 16, per = THREADS / lanes, j = threadIdx.x % lanes;
    const Vectors v = vectors_of(j, p.turn.R, INTER);
    const float inv_d = 1.f / static_cast<float>(p.D);
    const int heads = p.H + p.HK, units = n * heads;
    float qw[16], kw[16];
    load_weights(p.qw, v, qw);
    load_weights(p.kw, v, kw);
    for (int u0 = 0; u0 < units; u0 += per) {  // every lane makes the same number of steps (the shuffles need them all)
        const int u = u0 + threadIdx.x / lanes, tk = u / heads, hd = u - tk * heads;
        const bool live = u < units, is_q = hd < p.H;
        const long long tok = tok0 + tk;
        float a[8] = {}, b[8] = {}, w[16];
        const uint16_t *src = is_q ? p.q + tok * p.qs + hd * p.D : p.k + tok * p.ks + (hd - p.H) * p.D;
        if (live) {
            blk::unpack8(*reinterpret_cast<const uint4 *>(src + v.v0), a);
            blk::unpack8(*reinterpret_cast<const uint4 *>(src + v.v1), b);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = is_q ? qw[i] : kw[i];
        norm_and_turn<INTER>(a, b, p.hn.norm, p.hn.eps, inv_d, lanes, w, live && v.turned, table + tk * (p.turn.R / 2) + 8 * j);
        if (live) {
            uint16_t *dst = is_q ? p.qo + tok * p.qos + hd * p.D : p.ko + tok * p.kos + (hd - p.H) * p.D;
            *reinterpret_cast<uint4 *>(dst + v.v0) = blk::pack8(a);
            *reinterpret_cast<uint4 *>(dst + v.v1) = blk::pack8(b);
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
    int T, nseq, HK, D, tokens;
};

// Where a token's rows stand in the cache (of head 0), or -1 where it has none: positions below zero are padding.
__device__ __forceinline__ long long slot_of(const AppendParams &p, long long tok)
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
    return page * p.pages.stride + (pos & ((1 << p.pages.shift) - 1)) * p.D;
}

template <bool INTER>
__global__ void __launch_bounds__(THREADS) kda_kv_append_kernel(const AppendParams p)
{
    extern __shared__ float2 table[];
    __shared__ long long slots[32];
    const long long tok0 = static_cast<long long>(blockIdx.x) * p.tokens;
    const int n = static_cast<int>(min(static_cast<long long>(p.tokens), p.M - tok0));
    if (p.cu && blockIdx.x == 0) blk::check_bounds(p.cu, p.nseq, p.M);
    if (threadIdx.x < n) slots[threadIdx.x] = slot_of(p, tok0 + threadIdx.x);
    make_table(table, p.turn, tok0, n);
    __syncthreads();
    const int lanes = p.D / 16, per = THREADS / lanes, j = threadIdx.x % lanes;
    const Vectors v = vectors_of(j, p.turn.R, INTER);
    const float inv_d = 1.f / static_cast<float>(p.D);
    const long long page_size = 1LL << p.pages.shift, cache = (p.pages.count - 1) * p.pages.stride + p.HK * page_size * p.D;
    const int units = n * p.HK;
    float w[16];
    load_weights(p.kw, v, w);
    for (int u0 = 0; u0 < units; u0 += per) {
        const int u = u0 + threadIdx.x / lanes, tk = u / p.HK, hd = u - tk * p.HK;
        const long long tok = tok0 + tk, slot = u < units ? slots[tk] : -1;
        const bool live = slot >= 0;
        float a[8] = {}, b[8] = {};
        uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
        if (live) {
            const uint16_t *src = p.k + tok * p.ks + hd * p.D, *vsrc = p.v + tok * p.vs + hd * p.D;
            blk::unpack8(*reinterpret_cast<const uint4 *>(src + v.v0), a);
            blk::unpack8(*reinterpret_cast<const uint4 *>(src + v.v1), b);
            v0 = *reinterpret_cast<const uint4 *>(vsrc + v.v0);
            v1 = *reinterpret_cast<const uint4 *>(vsrc + v.v1);
        }
        norm_and_turn<INTER>(a, b, p.hn.norm, p.hn.eps, inv_d, lanes, w, live && v.turned, table + tk * (p.turn.R / 2) + 8 * j);
        const long long dst = slot + hd * page_size * p.D;
        if (live && gmem_ok(dst, p.D, cache)) {
            *reinterpret_cast<uint4 *>(p.kc + dst + v.v0) = blk::pack8(a);
            *reinterpret_cast<uint4 *>(p.kc + dst + v.v1) = blk::pack8(b);
            *reinterpret_cast<uint4 *>(p.vc + dst + v.v0) = v0;
            *reinterpret_cast<uint4 *>(p.vc + dst + v.v1) = v1;
        }
    }
}

}  // namespace rope
}  // namespace kda
