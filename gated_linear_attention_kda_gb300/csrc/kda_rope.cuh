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
constexpr int BATCH = 4;       // heads of a lane group in flight
constexpr int MAX_TOKENS = 16; // of a CTA

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

__device__ __forceinline__ void load8s(const float *p, float (&f)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// A lane owns two vectors of eight channels of a head, of the part that is turned both members of eight pairs. First and
// second vectors of neighbouring lanes are neighbours, so that an access covers whole sectors (32,768 tokens of 20 heads
// of 128, 32 channels turned: 51 us so, 78 us with a lane's vectors side by side).
struct Vectors {
    int v0, v1;    // first channel of either
    int c0, c1;    // first pair of either in the token's table (interleaved pairs; else c0 is both's)
    bool t0, t1;   // turned
};
template <bool INTER>
__device__ __forceinline__ Vectors vectors_of(int j, int lanes, int R)
{
    if (INTER) return {8 * j, 8 * (j + lanes), 4 * j, 4 * (j + lanes), 8 * j < R, 8 * (j + lanes) < R};
    const int half = R / 16;  // vectors in half of the turned part
    if (j < half) return {8 * j, 8 * (j + half), 8 * j, 8 * j, true, true};
    return {8 * (j + half), 8 * (j + lanes), 0, 0, false, false};
}

// Norm and turn of one head held by `lanes` neighbouring lanes; w: the head's weights or NULL; cs: the token's turns.
template <bool INTER>
__device__ __forceinline__ void norm_and_turn(float (&a)[8], float (&b)[8], bool norm, float eps, float inv_d, int lanes, const float *w,
                                              const Vectors &v, const float2 *cs)
{
    if (norm) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            ss = ffma2(make_float2(a[i], a[i + 1]), make_float2(a[i], a[i + 1]), ss);
            ss = ffma2(make_float2(b[i], b[i + 1]), make_float2(b[i], b[i + 1]), ss);
        }
        float sum = ss.x + ss.y;
        for (int m = lanes >> 1; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const float f = rsqrtf(fmaf(sum, inv_d, eps));
        float wa[8], wb[8];
        load8s(w + v.v0, wa);
        load8s(w + v.v1, wb);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] *= f * wa[i];
            b[i] *= f * wb[i];
        }
    }
    if (INTER) {  // pairs inside the vectors
        auto turn = [&](float(&x)[8], int c) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 t = cs[c + i / 2];
                const float y = x[i];
                x[i] = y * t.x - x[i + 1] * t.y;
                x[i + 1] = x[i + 1] * t.x + y * t.y;
            }
        };
        if (v.t0) turn(a, v.c0);
        if (v.t1) turn(b, v.c1);
    } else if (v.t0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 t = cs[v.c0 + i];
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

// A head's weights in shared memory (1 where there are none).
__device__ __forceinline__ void keep_weights(float *dst, const float *w, int D)
{
    for (int i = threadIdx.x; i < D; i += blockDim.x) dst[i] = w ? __ldg(w + i) : 1.f;
}

// (token of the CTA, head) of a lane group, walked along without dividing
struct Item {
    int tk, hd;
    __device__ __forceinline__ void next(int by, int heads)
    {
        hd += by;
        while (hd >= heads) {
            hd -= heads;
            ++tk;
        }
    }
};

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
    __shared__ __align__(16) float weights[2][MAX_D];
    const long long tok0 = static_cast<long long>(blockIdx.x) * p.tokens;
    const int n = static_cast<int>(min(static_cast<long long>(p.tokens), p.M - tok0));
    const int lanes = p.D / 16, per = THREADS / lanes, j = threadIdx.x % lanes, heads = p.H + p.HK, units = n * heads;
    const Vectors v = vectors_of<INTER>(j, lanes, p.turn.R);
    const float inv_d = 1.f / static_cast<float>(p.D);
    Item ld = {0, 0}, st;
    ld.next(static_cast<int>(threadIdx.x) / lanes, heads);
    st = ld;
    uint4 x[BATCH][2];
    auto fetch = [&]() {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            x[b][0] = x[b][1] = make_uint4(0u, 0u, 0u, 0u);
            if (ld.tk < n) {
                const bool is_q = ld.hd < p.H;
                const long long at = is_q ? (tok0 + ld.tk) * p.qs + ld.hd * p.D : (tok0 + ld.tk) * p.ks + (ld.hd - p.H) * p.D;
                const uint16_t *src = is_q ? p.q : p.k;
                if (gmem_ok(at, p.D, is_q ? (p.M - 1) * p.qs + p.H * p.D : (p.M - 1) * p.ks + p.HK * p.D)) {
                    x[b][0] = *reinterpret_cast<const uint4 *>(src + at + v.v0);
                    x[b][1] = *reinterpret_cast<const uint4 *>(src + at + v.v1);
                }
            }
            ld.next(per, heads);
        }
    };
    fetch();  // ahead of the table, whose chain is long
    make_table(table, p.turn, tok0, n);
    if (p.hn.norm) {
        keep_weights(weights[0], p.qw, p.D);
        keep_weights(weights[1], p.kw, p.D);
    }
    __syncthreads();
    for (int u0 = 0; u0 < units; u0 += per * BATCH) {  // every lane makes the same number of steps (the shuffles need them all)
        if (u0 > 0) fetch();
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const bool live = st.tk < n, is_q = st.hd < p.H;
            float f[8], g[8];
            blk::unpack8(x[b][0], f);
            blk::unpack8(x[b][1], g);
            norm_and_turn<INTER>(f, g, p.hn.norm, p.hn.eps, inv_d, lanes, weights[is_q ? 0 : 1], v,
                                 table + (live ? st.tk : 0) * (p.turn.R / 2));
            if (live) {
                const long long at = is_q ? (tok0 + st.tk) * p.qos + st.hd * p.D : (tok0 + st.tk) * p.kos + (st.hd - p.H) * p.D;
                uint16_t *dst = is_q ? p.qo : p.ko;
                if (gmem_ok(at, p.D, is_q ? (p.M - 1) * p.qos + p.H * p.D : (p.M - 1) * p.kos + p.HK * p.D)) {
                    *reinterpret_cast<uint4 *>(dst + at + v.v0) = blk::pack8(f);
                    *reinterpret_cast<uint4 *>(dst + at + v.v1) = blk::pack8(g);
                }
            }
            st.next(per, heads);
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
    __shared__ __align__(16) float weights[MAX_D];
    __shared__ long long slots[MAX_TOKENS];
    constexpr int B = BATCH / 2;  // keys and values
    const long long tok0 = static_cast<long long>(blockIdx.x) * p.tokens;
    const int n = static_cast<int>(min(static_cast<long long>(p.tokens), p.M - tok0));
    if (p.cu && blockIdx.x == 0) blk::check_bounds(p.cu, p.nseq, p.M);
    const int lanes = p.D / 16, per = THREADS / lanes, j = threadIdx.x % lanes, units = n * p.HK;
    const Vectors v = vectors_of<INTER>(j, lanes, p.turn.R);
    const float inv_d = 1.f / static_cast<float>(p.D);
    const long long page_size = 1LL << p.pages.shift, cache = (p.pages.count - 1) * p.pages.stride + p.HK * page_size * p.D;
    Item ld = {0, 0}, st;
    ld.next(static_cast<int>(threadIdx.x) / lanes, p.HK);
    st = ld;
    uint4 x[B][2], y[B][2];
    auto fetch = [&]() {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            x[b][0] = x[b][1] = y[b][0] = y[b][1] = make_uint4(0u, 0u, 0u, 0u);
            if (ld.tk < n) {
                const long long at = (tok0 + ld.tk) * p.ks + ld.hd * p.D, vat = (tok0 + ld.tk) * p.vs + ld.hd * p.D;
                if (gmem_ok(at, p.D, (p.M - 1) * p.ks + p.HK * p.D) && gmem_ok(vat, p.D, (p.M - 1) * p.vs + p.HK * p.D)) {
                    x[b][0] = *reinterpret_cast<const uint4 *>(p.k + at + v.v0);
                    x[b][1] = *reinterpret_cast<const uint4 *>(p.k + at + v.v1);
                    y[b][0] = *reinterpret_cast<const uint4 *>(p.v + vat + v.v0);
                    y[b][1] = *reinterpret_cast<const uint4 *>(p.v + vat + v.v1);
                }
            }
            ld.next(per, p.HK);
        }
    };
    fetch();  // ahead of the table and the look-up of pages, whose chains are long
    if (threadIdx.x < n) slots[threadIdx.x] = slot_of(p, tok0 + threadIdx.x);
    make_table(table, p.turn, tok0, n);
    if (p.hn.norm) keep_weights(weights, p.kw, p.D);
    __syncthreads();
    for (int u0 = 0; u0 < units; u0 += per * B) {
        if (u0 > 0) fetch();
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const long long slot = st.tk < n ? slots[st.tk] : -1;
            float f[8], g[8];
            blk::unpack8(x[b][0], f);
            blk::unpack8(x[b][1], g);
            norm_and_turn<INTER>(f, g, p.hn.norm, p.hn.eps, inv_d, lanes, weights, v,
                                 table + (st.tk < n ? st.tk : 0) * (p.turn.R / 2));
            const long long dst = slot + st.hd * page_size * p.D;
            if (slot >= 0 && gmem_ok(dst, p.D, cache)) {
                *reinterpret_cast<uint4 *>(p.kc + dst + v.v0) = blk::pack8(f);
                *reinterpret_cast<uint4 *>(p.kc + dst + v.v1) = blk::pack8(g);
                *reinterpret_cast<uint4 *>(p.vc + dst + v.v0) = y[b][0];
                *reinterpret_cast<uint4 *>(p.vc + dst + v.v1) = y[b][1];
            }
            st.next(per, p.HK);
        }
    }
}

}  // namespace rope
}  // namespace kda
