// kda_conv.cuh -- short causal convolution along the tokens (W = 2, 3 or 4 taps per channel), for
// packed or batched prompts and for single tokens:
//   u[t, c] = bias[c] + sum_{j < W} weight[c, j] x[t - (W - 1) + j, c],   out = u or u sigmoid(u)
// with the rows of the initial state (or zeros) before a sequence's first token.
//
// HBM-bound: 2 bytes in and 2 out per element against W FMAs and one sigmoid. A thread owns eight
// channels (one 16-byte access per token) and walks a run of tokens of them with the last W - 1 rows in
// registers, so a row is read once per run plus the W - 1 rows before it; the BATCH rows of the next
// step are loaded before those of the present one are filtered. Arithmetic is in fp32 pairs.
// Four taps with SiLU: 8 x 4096 tokens of 2048 channels 49.9 us (5.4 TB/s), 16 packed prompts, 65,519 tokens in all,
// 4352 channels 188 us (6.1 TB/s; a plain copy makes 6.7). Warps wait for loads (long scoreboard) more than for
// anything else; the sigmoid's two approximations per element take 30 % of their pipe.
#pragma once
#include "blk_common.cuh"

namespace kda {
namespace conv {

constexpr int THREADS = 128;
constexpr int BLOCKS = 4;    // resident CTAs per SM (five spill: 95 us where four take 55)
constexpr int RUN_COST = 8;  // what starting a run costs, in tokens
constexpr int MAX_RUN = 256; // tokens per thread at most
constexpr int BATCH = 4;     // rows in flight per thread (eight, at three CTAs per SM: 68 us)

struct ConvParams {
    const uint16_t *x, *init;
    uint16_t *out, *fin;
    const float *weight, *bias;
    const int64_t *cu;
    long long xs, os;       // elements between tokens
    long long total, T;     // tokens in all, per batch row
    long long tiles;        // blocks of the token axis (the blocks after them write final states)
    int nseq, C, act;
    int cg;                 // threads along the channels (a power of two <= THREADS)
    int run;                // tokens per thread
};

// Eight channels of a token row, `stride` elements apart, lie in a tensor of `rows` rows (the checked build looks).
__device__ __forceinline__ bool row_ok(long long row, int c, long long rows, long long stride, int C)
{
    return gmem_ok(static_cast<size_t>(row * stride + c), 8, static_cast<size_t>((rows - 1) * stride + C));
}

// Eight channels as four pairs (paired fp32 arithmetic).
struct Row {
    float2 v[4];
};
__device__ __forceinline__ Row unpack(const uint4 &r)
{
    return {{make_float2(bf16_lo(r.x), bf16_hi(r.x)), make_float2(bf16_lo(r.y), bf16_hi(r.y)),
             make_float2(bf16_lo(r.z), bf16_hi(r.z)), make_float2(bf16_lo(r.w), bf16_hi(r.w))}};
}

template <int W>
struct Taps {
    Row w[W], b;
    __device__ __forceinline__ void load(const float *weight, const float *bias, int c)
    {
        float buf[8 * W];  // the eight channels' taps, contiguous
        const float4 *src = reinterpret_cast<const float4 *>(weight + static_cast<size_t>(c) * W);
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) {
            const float4 q = __ldg(src + i);
            buf[4 * i] = q.x; buf[4 * i + 1] = q.y; buf[4 * i + 2] = q.z; buf[4 * i + 3] = q.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j].v[i] = make_float2(buf[2 * i * W + j], buf[(2 * i + 1) * W + j]);
            b.v[i] = bias ? __ldg(reinterpret_cast<const float2 *>(bias + c) + i) : make_float2(0.f, 0.f);
        }
    }
    // One output row from the W rows that end with it.
    __device__ __forceinline__ uint4 row(const Row *f, bool silu) const
    {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 u = b.v[i];
#pragma unroll
            for (int j = 0; j < W; ++j) u = ffma2(w[j].v[i], f[j].v[i], u);
            if (silu) u = fmul2(u, blk::sigmoid_fast2(u));
            o[i] = pack_bf16(u.x, u.y);
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
};

// The last W - 1 rows of [initial state ; x] of one sequence, eight channels. All rows are read
// before any is written: the final state may be the initial state's buffer.
template <int W>
__device__ __forceinline__ void write_final(const ConvParams &p, int seq, int c)
{
    long long b, len;
    if (p.cu) {
        b = p.cu[seq];
        const long long e = p.cu[seq + 1];
        if (b < 0 || e < b || e > p.total) return;
        len = e - b;
    } else {
        b = static_cast<long long>(seq) * p.T;
        len = p.T;
    }
    const size_t st = static_cast<size_t>(seq) * (W - 1) * p.C + c;
    const size_t st_elems = static_cast<size_t>(p.nseq) * (W - 1) * p.C;
    uint4 row[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const long long at = len + j;  // row of [init ; x]
        row[j] = make_uint4(0u, 0u, 0u, 0u);
        if (at >= W - 1) {
            if (row_ok(b + at - (W - 1), c, p.total, p.xs, p.C)) row[j] = *reinterpret_cast<const uint4 *>(p.x + (b + at - (W - 1)) * p.xs + c);
        } else if (p.init && gmem_ok(st + at * p.C, 8, st_elems))
            row[j] = *reinterpret_cast<const uint4 *>(p.init + st + at * p.C);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        if (gmem_ok(st + static_cast<size_t>(j) * p.C, 8, st_elems))
            *reinterpret_cast<uint4 *>(p.fin + st + static_cast<size_t>(j) * p.C) = row[j];
}

template <int W>
__global__ void __launch_bounds__(THREADS, BLOCKS) kda_conv_kernel(const ConvParams p)
{
    if (p.cu && blockIdx.x == 0 && blockIdx.y == 0) blk::check_bounds(p.cu, p.nseq, p.total);
    const int nc8 = p.C >> 3;
    if (blockIdx.x >= p.tiles) {  // final states, one thread per (sequence, eight channels)
        if (blockIdx.y || !p.fin) return;
        const long long i = (static_cast<long long>(blockIdx.x) - p.tiles) * THREADS + threadIdx.x;
        if (i < static_cast<long long>(p.nseq) * nc8)
            write_final<W>(p, static_cast<int>(i / nc8), static_cast<int>(i % nc8) * 8);
        return;
    }
    const int c8 = blockIdx.y * p.cg + (threadIdx.x & (p.cg - 1));
    if (c8 >= nc8) return;
    const int c = 8 * c8, tg = THREADS / p.cg;
    long long t = (static_cast<long long>(blockIdx.x) * tg + threadIdx.x / p.cg) * p.run;
    const long long t_end = min(t + p.run, p.total);
    Taps<W> taps;
    taps.load(p.weight, p.bias, c);
    const bool silu = p.act == KDA_ACT_SILU;
    while (t < t_end) {
        blk::Enclosing sq;
        if (p.cu) {
            sq = blk::find_sequence(p.cu, p.nseq, p.total, t);
            if (!sq.ok) {  // a token of no sequence: bad bounds, flagged above
                ++t;
                continue;
            }
        } else {
            sq.seq = static_cast<int>(t / p.T);
            sq.b = sq.seq * p.T;
            sq.e = sq.b + p.T;
        }
        const long long end = min(sq.e, t_end);
        const uint16_t *src = p.x + t * p.xs + c;
        uint16_t *dst = p.out + t * p.os + c;
        int n = static_cast<int>(end - t);  // tokens of this sequence in the run
        long long tok = t;                  // of src and dst
        uint4 raw[BATCH];
        auto fetch = [&] {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                raw[i] = make_uint4(0u, 0u, 0u, 0u);
                if (i < n && row_ok(tok + i, c, p.total, p.xs, p.C)) raw[i] = __ldg(reinterpret_cast<const uint4 *>(src + i * p.xs));
            }
        };
        fetch();
        Row f[W - 1 + BATCH];  // the W - 1 rows before the batch, and the batch
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const long long at = t - (W - 1) + j;
            uint4 r = make_uint4(0u, 0u, 0u, 0u);
            if (at >= sq.b) {
                if (row_ok(at, c, p.total, p.xs, p.C)) r = __ldg(reinterpret_cast<const uint4 *>(p.x + at * p.xs + c));
            } else if (p.init) {
                const size_t st = (static_cast<size_t>(sq.seq) * (W - 1) + static_cast<size_t>(at - sq.b + (W - 1))) * p.C + c;
                if (gmem_ok(st, 8, static_cast<size_t>(p.nseq) * (W - 1) * p.C)) r = *reinterpret_cast<const uint4 *>(p.init + st);
            }
            f[j] = unpack(r);
        }
#pragma unroll 1
        while (n > 0) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) f[W - 1 + i] = unpack(raw[i]);
            const int m = n;
            n -= BATCH;
            src += BATCH * p.xs;
            tok += BATCH;
            fetch();  // the next batch's rows are in flight while this one is filtered
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (i < m && row_ok(tok - BATCH + i, c, p.total, p.os, p.C)) *reinterpret_cast<uint4 *>(dst + i * p.os) = taps.row(f + i, silu);
            dst += BATCH * p.os;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) f[j] = f[BATCH + j];
        }
        t = end;
    }
}

// One token of S sequences. A thread owns eight channels of STEP_SEQS sequences (it reads the taps once
// for all of them; 128 sequences x 6144 channels: 3.9 us on the device, 14.8 us with one sequence per thread
// and scalar tap loads). All rows of a sequence are read before its state or output is written: out may be x.
constexpr int STEP_SEQS = 4;
template <int W>
__global__ void __launch_bounds__(THREADS) kda_conv_step_kernel(const ConvParams p, uint16_t *state)
{
    const int nc8 = p.C >> 3;
    const long long i = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
    const long long s0 = i / nc8 * STEP_SEQS;
    if (s0 >= p.nseq) return;
    const int c = static_cast<int>(i % nc8) * 8;
    uint16_t *st = state + s0 * (W - 1) * p.C + c;
    auto st_ok = [&](int k, int j) { return gmem_ok(static_cast<size_t>((s0 + k) * (W - 1) + j) * p.C + c, 8, static_cast<size_t>(p.nseq) * (W - 1) * p.C); };
    uint4 raw[STEP_SEQS][W] = {};
#pragma unroll
    for (int k = 0; k < STEP_SEQS; ++k)
        if (s0 + k < p.nseq) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                if (st_ok(k, j)) raw[k][j] = *reinterpret_cast<const uint4 *>(st + static_cast<size_t>(k * (W - 1) + j) * p.C);
            if (row_ok(s0 + k, c, p.nseq, p.xs, p.C)) raw[k][W - 1] = *reinterpret_cast<const uint4 *>(p.x + (s0 + k) * p.xs + c);
        }
    Taps<W> taps;
    taps.load(p.weight, p.bias, c);
#pragma unroll
    for (int k = 0; k < STEP_SEQS; ++k)
        if (s0 + k < p.nseq) {
            Row f[W];
#pragma unroll
            for (int j = 0; j < W; ++j) f[j] = unpack(raw[k][j]);
            if (row_ok(s0 + k, c, p.nseq, p.os, p.C)) *reinterpret_cast<uint4 *>(p.out + (s0 + k) * p.os + c) = taps.row(f, p.act == KDA_ACT_SILU);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                if (st_ok(k, j)) *reinterpret_cast<uint4 *>(st + static_cast<size_t>(k * (W - 1) + j) * p.C) = raw[k][j + 1];
        }
}

}  // namespace conv
}  // namespace kda
