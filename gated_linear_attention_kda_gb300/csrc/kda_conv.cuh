// kda_conv.cuh -- short causal convolution along the tokens (W = 2, 3 or 4 taps per channel), for
// packed or batched prompts and for single tokens:
//   u[t, c] = bias[c] + sum_{j < W} weight[c, j] x[t - (W - 1) + j, c],   out = u or u sigmoid(u)
// with the rows of the initial state (or zeros) before a sequence's first token.
//
// HBM-bound: 2 bytes in and 2 out per element against W FMAs and one sigmoid. A thread owns eight
// channels (one 16-byte access per token) and walks RUN tokens of them with the last W - 1 rows in
// registers, so a row is read once per run plus the W - 1 rows before it; BATCH rows are loaded
// before any is used, which keeps the loads of a whole batch in flight.
#pragma once
#include "blk_common.cuh"

namespace kda {
namespace conv {

constexpr int THREADS = 128;
constexpr int RUN = 32;    // tokens per thread
constexpr int BATCH = 4;   // rows in flight per thread

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
};

template <int W>
__device__ __forceinline__ void load_weights(const float *weight, const float *bias, int c, float (&w)[W][8], float (&b)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = __ldg(weight + static_cast<size_t>(c + i) * W + j);
        b[i] = bias ? __ldg(bias + c + i) : 0.f;
    }
}

// One output row from the W rows that end with it.
template <int W>
__device__ __forceinline__ uint4 filter_row(const float (*f)[8], const float (&w)[W][8], const float (&b)[8], int act)
{
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u[i] = b[i];
#pragma unroll
        for (int j = 0; j < W; ++j) u[i] = fmaf(w[j][i], f[j][i], u[i]);
        u[i] = blk::apply_act(u[i], act);
    }
    return blk::pack8(u);
}

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
        if (at >= W - 1)
            row[j] = *reinterpret_cast<const uint4 *>(p.x + (b + at - (W - 1)) * p.xs + c);
        else if (p.init && gmem_ok(st + at * p.C, 8, st_elems))
            row[j] = *reinterpret_cast<const uint4 *>(p.init + st + at * p.C);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        if (gmem_ok(st + static_cast<size_t>(j) * p.C, 8, st_elems))
            *reinterpret_cast<uint4 *>(p.fin + st + static_cast<size_t>(j) * p.C) = row[j];
}

template <int W>
__global__ void __launch_bounds__(THREADS) kda_conv_kernel(const ConvParams p)
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
    long long t = (static_cast<long long>(blockIdx.x) * tg + threadIdx.x / p.cg) * RUN;
    const long long t_end = min(t + RUN, p.total);
    float w[W][8], bias[8];
    load_weights<W>(p.weight, p.bias, c, w, bias);
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
        float f[W - 1 + BATCH][8];  // rows t - (W - 1) .. t + BATCH - 1
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const long long at = t - (W - 1) + j;
            uint4 r = make_uint4(0u, 0u, 0u, 0u);
            if (at >= sq.b)
                r = __ldg(reinterpret_cast<const uint4 *>(p.x + at * p.xs + c));
            else if (p.init)
                r = *reinterpret_cast<const uint4 *>(
                    p.init + (static_cast<size_t>(sq.seq) * (W - 1) + static_cast<size_t>(at - sq.b + (W - 1))) * p.C + c);
            blk::unpack8(r, f[j]);
        }
        for (; t < end; t += BATCH) {
            uint4 raw[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                raw[i] = make_uint4(0u, 0u, 0u, 0u);
                if (t + i < end) raw[i] = __ldg(reinterpret_cast<const uint4 *>(p.x + (t + i) * p.xs + c));
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) blk::unpack8(raw[i], f[W - 1 + i]);
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (t + i < end) *reinterpret_cast<uint4 *>(p.out + (t + i) * p.os + c) = filter_row<W>(f + i, w, bias, p.act);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) f[j][i] = f[BATCH + j][i];
        }
        t = end;
    }
}

// One token of S sequences: a thread holds eight channels of one sequence, all rows read first
// (out may be x), and shifts the state by one row. Launch latency bounds it.
template <int W>
__global__ void __launch_bounds__(THREADS) kda_conv_step_kernel(const ConvParams p, uint16_t *state)
{
    const int nc8 = p.C >> 3;
    const long long i = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
    if (i >= static_cast<long long>(p.nseq) * nc8) return;
    const long long s = i / nc8;
    const int c = static_cast<int>(i % nc8) * 8;
    uint16_t *st = state + s * (W - 1) * p.C + c;
    uint4 raw[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[j] = *reinterpret_cast<const uint4 *>(st + static_cast<size_t>(j) * p.C);
    raw[W - 1] = *reinterpret_cast<const uint4 *>(p.x + s * p.xs + c);
    float w[W][8], bias[8], f[W][8];
    load_weights<W>(p.weight, p.bias, c, w, bias);
#pragma unroll
    for (int j = 0; j < W; ++j) blk::unpack8(raw[j], f[j]);
    *reinterpret_cast<uint4 *>(p.out + s * p.os + c) = filter_row<W>(f, w, bias, p.act);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) *reinterpret_cast<uint4 *>(st + static_cast<size_t>(j) * p.C) = raw[j + 1];
}

}  // namespace conv
}  // namespace kda
