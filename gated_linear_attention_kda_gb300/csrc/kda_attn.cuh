// kda_attn.cuh -- softmax attention of one new token per sequence over a paged cache of keys and values.
//   out = softmax(scale q K^T) V over the cached positions 0 .. position
// Bound by HBM: a cached key and value are read once for the query heads that share them, which are the rows of the
// warp MMAs (up to 16; more in further units). The cache is cut into slices of 16 tokens, ordered by sequence, key head
// and position, and the warps of a grid that fills the machine take equal runs of slices, whatever the lengths: a unit
// (a sequence's key head) that lies inside one run is finished there, the parts of the others go to the workspace
// and are joined by a second kernel. A run is read by its warp alone (no barrier in the loop): cp.async into a ring of
// its own, the scores of 16 tokens in registers, one pass with the running maximum and sum of the softmax. What stands
// behind a sequence's end is not read: its rows are filled with zeros on the way.
// Measured (device): 128 sequences of some 4,100 tokens, 4 key heads of 128, 1.07 GB: 174 us, 6.2 TB/s; one sequence of
// 131,072 tokens, 8 key heads, .54 GB: 90 us, 5.9 TB/s; 8 sequences of 4,001 in all, 2 key heads of 64: 7.9 us, where the
// cache is in L2 and the two launches and the chain of positions, table, pages and slices bound it.
// Without a workspace a unit is one warp's, three slices of 8 KB in flight: 7.4 ms for the 131,072 tokens, 298 us for 128
// sequences of 4,096 (184 with one, per call). Above 16 query heads per key head every further 16 read the cache again: 128
// sequences of 4,096 with one key head take 64 us for 16 query heads, 99 for 20, 169 for 64.
#pragma once
#include "kda_rope.cuh"

namespace kda {
namespace attn {

using rope::Pages;

constexpr int WARPS = 4;        // of a CTA; each works alone
constexpr int THREADS = 32 * WARPS;
constexpr int SL = 16;          // tokens of a slice
constexpr int CTAS = 2;         // per SM
constexpr int JOIN_THREADS = 256;
constexpr float LOWEST = -3.402823466e38f;  // the least number

struct AttnParams {
    const uint16_t *q, *kc, *vc;
    uint16_t *out;
    float *lse;                 // [S, H] or NULL
    long long qs, os;           // elements between sequences
    const int64_t *positions;   // of the new tokens
    Pages pages;
    float scale;
    int S, H, HK, D;
    int rows, tiles;            // query heads per key head, and row tiles of 16 of them
    int workers;                // warps with a run
    float *ws;                  // parts: [workers][2][16][D], then their maxima and sums [workers][2][16][2]; NULL: units are not cut
};

__host__ __device__ constexpr int stages_of(int D) { return D == 128 ? 3 : 6; }
__host__ __device__ constexpr int slice_bytes(int D) { return 2 * SL * 2 * D; }  // keys, then values
__host__ __device__ constexpr int smem_of(int D) { return WARPS * stages_of(D) * slice_bytes(D); }

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
__device__ __forceinline__ long long slices_of(long long tokens) { return (tokens + SL - 1) / SL; }

__device__ __forceinline__ long long warp_sum(long long v)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// Slices of the sequences before `seq` (one per key head and row tile), by a whole warp.
__device__ __forceinline__ long long slices_before(const AttnParams &p, int seq)
{
    long long n = 0;
    for (int s = threadIdx.x & 31; s < seq; s += 32) n += slices_of(tokens_of(p, s));
    return warp_sum(n);
}

// Quotient of numbers that nearly always have 32 bits (the 64-bit division takes some hundred instructions).
__device__ __forceinline__ long long quotient(long long a, long long b)
{
    return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// The runs of `total` slices: as many as there are warps, but none shorter than MIN_RUN, and their first slices.
constexpr int MIN_RUN = 2;  // 7.9 us at the small case above; 4: 9.4, 8: 12.2
struct Runs {
    long long total, each;
    uint32_t count, rest;
    __device__ __forceinline__ Runs(const AttnParams &p, long long total_) : total(total_)
    {
        count = static_cast<uint32_t>(min(max(total / MIN_RUN, 1LL), static_cast<long long>(p.workers)));
        each = quotient(total, count);
        rest = static_cast<uint32_t>(total - each * count);
    }
    // (workers are a few thousand: the product fits)
    __device__ __forceinline__ long long start(uint32_t w) const { return each * w + rest * w / count; }
    // the run that holds slice x
    __device__ __forceinline__ uint32_t of(long long x) const
    {
        // nearly: a float's rounding is off by less than one of a few thousand runs
        uint32_t w = min(static_cast<uint32_t>(__fdividef(static_cast<float>(x) * static_cast<float>(count), static_cast<float>(total))), count - 1);
        while (w > 0 && start(w) > x) --w;
        while (w + 1 < count && start(w + 1) <= x) ++w;
        return w;
    }
};
// Where slice x stands: sequence, unit of it, slice of the unit; by a whole warp.
struct Place {
    int seq, unit;
    long long slice, slices, tokens;
    // the next slice; past a sequence's last unit, the next sequence that has tokens
    __device__ __forceinline__ bool next(const AttnParams &p)  // true where a unit begins
    {
        if (++slice < slices) return false;
        slice = 0;
        if (++unit < p.HK * p.tiles) return true;
        unit = 0;
        slices = 0;
        while (slices == 0 && ++seq < p.S) {
            tokens = tokens_of(p, seq);
            slices = slices_of(tokens);
        }
        return true;
    }
};
__device__ __forceinline__ Place locate(const AttnParams &p, long long x)
{
    const int lane = threadIdx.x & 31, units = p.HK * p.tiles;
    long long before = 0;
    for (int s0 = 0; s0 < p.S; s0 += 32) {
        const long long t = s0 + lane < p.S ? tokens_of(p, s0 + lane) : 0, n = slices_of(t) * units;
        long long inc = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, inc, m);
            if (lane >= m) inc += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, x < before + inc);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const long long at = x - before - __shfl_sync(0xffffffffu, inc - n, src), tokens = __shfl_sync(0xffffffffu, t, src), sl = slices_of(tokens);
            const long long unit = quotient(at, sl);
            return {s0 + src, static_cast<int>(unit), at - unit * sl, sl, tokens};
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    return {p.S, 0, 0, 0, 0};
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live)
{
    if (!smem_ok(dst, 16)) return;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D>
__global__ void __launch_bounds__(THREADS, CTAS) kda_attn_step_kernel(const AttnParams p)
{
    constexpr int STAGES = stages_of(D), SLICE = slice_bytes(D), ROW = 2 * D, CH = D / 8;  // CH: vectors of 16 bytes in a row
    extern __shared__ uint8_t smem_dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
    const uint32_t ring = smem_u32(smem_dyn) + warp * (STAGES * SLICE);
    // sequences that see nothing
    for (int s = blockIdx.x; s < p.S; s += gridDim.x)
        if (tokens_of(p, s) == 0) {
            for (int i = threadIdx.x; i < p.H * CH; i += THREADS) reinterpret_cast<uint4 *>(p.out + s * p.os)[i] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse)
                for (int i = threadIdx.x; i < p.H; i += THREADS) p.lse[static_cast<long long>(s) * p.H + i] = -INFINITY;
        }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may wait in place
    const uint32_t worker = blockIdx.x * WARPS + warp;
    const Runs runs(p, slices_before(p, p.S) * p.HK * p.tiles);
    if (worker >= runs.count) return;
    long long x0 = runs.start(worker), x1 = runs.start(worker + 1);
    if (x0 >= x1) return;
    Place at = locate(p, x0);
    if (!p.ws) {  // whole units: those that begin inside the run
        if (at.slice) {
            x0 += at.slices - at.slice;
            at.slice = at.slices - 1;
            at.next(p);
        }
        if (x0 >= x1) return;
        const Place last = locate(p, x1 - 1);
        x1 += last.slices - 1 - last.slice;
    }
    const long long page_size = 1LL << p.pages.shift;
    const size_t cache = static_cast<size_t>(p.pages.count - 1) * p.pages.stride + static_cast<size_t>(p.HK) * page_size * D;
    // the page of eight tokens of a place (a slice lies in one page, or in two of eight)
    auto page_of = [&](const Place &pl, int half) -> int {
        const long long t = pl.slice * SL + 8 * half;
        if (pl.seq >= p.S || t >= pl.tokens) return -2;  // nothing there
        const int page = __ldg(p.pages.table + static_cast<long long>(pl.seq) * p.pages.width + (t >> p.pages.shift));
        return page < 0 ? -1 : page;
    };
    Place ld = at;       // the next slice to be asked for; its pages are looked up one slice ahead
    int pg[2] = {page_of(ld, 0), page_of(ld, 1)};
    int ask = 0, st_ld = 0;
    unsigned bad = 0u;   // which half slices in the ring stand on pages that do not exist, two bits a buffer
    const int count = static_cast<int>(x1 - x0);  // slices of the run
    auto load = [&]() {
        const uint32_t dst = ring + st_ld * SLICE;
        const int hk = ld.unit / p.tiles;
        const long long t0 = ld.slice * SL;
        const int c = lane % CH;
        const unsigned b = (pg[0] != -2 && (pg[0] < 0 || pg[0] >= p.pages.count) ? 1u : 0u) | (pg[1] != -2 && (pg[1] < 0 || pg[1] >= p.pages.count) ? 2u : 0u);
        if (b && lane == 0) atomicOr(&g_dev_error, DEVERR_PAGES);
        bad = (bad & ~(3u << 2 * st_ld)) | b << 2 * st_ld;
#pragma unroll
        for (int i = 0; i < SL * CH / 32; ++i) {
            const int r = lane / CH + (32 / CH) * i;
            const int page = r < 8 ? pg[0] : pg[1];
            const long long t = t0 + r;
            const bool live = t < ld.tokens && page >= 0 && page < p.pages.count;
            const long long e = live ? page * p.pages.stride + (hk * page_size + (t & (page_size - 1))) * D + 8 * c : 0;
            const bool ok = live && gmem_ok(e, 8, cache);
            const uint32_t o = dst + r * ROW + ((c ^ (r & 7)) << 4);
            cp_async16(o, p.kc + e, ok);
            cp_async16(o + SL * ROW, p.vc + e, ok);
        }
        st_ld = st_ld + 1 == STAGES ? 0 : st_ld + 1;
        ld.next(p);
        pg[0] = page_of(ld, 0);
        pg[1] = page_of(ld, 1);
    };
    for (; ask < STAGES - 1; ++ask) {
        if (ask < count) load();
        cp_commit();
    }

    const float c2 = p.scale * LOG2E;
    uint32_t qa[D / 16][4];
    float acc[D / 8][4], top[2], sum[2];
    unsigned seen;  // tokens that count, of the unit's slices so far
    auto begin = [&]() {  // queries of a unit's rows, and nothing seen so far
        const int hk = at.unit / p.tiles, r0 = (at.unit - hk * p.tiles) * 16;
        const uint16_t *qp = p.q + at.seq * p.qs + (static_cast<long long>(hk) * p.rows + r0) * D + 2 * t4;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = g8 + 8 * (j & 1);
                qa[k][j] = r0 + r < p.rows ? __ldg(reinterpret_cast<const uint32_t *>(qp + r * D + 16 * k + 8 * (j >> 1))) : 0u;
            }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        top[0] = top[1] = -INFINITY;
        sum[0] = sum[1] = 0.f;
        seen = 0u;
    };
    begin();
    bool whole = at.slice == 0;  // the unit's first slice is in this run
    int st = 0;
    for (int i = 0; i < count; ++i) {
        if (ask < count) load();
        ++ask;
        cp_commit();
        cp_wait<STAGES - 1>();
        __syncwarp();
        const uint32_t kb = ring + st * SLICE, vb = kb + SL * ROW;
        // which of the slice's tokens count: those up to the position, on pages that exist
        unsigned live = 0xffffu;
        if (at.slice * SL + SL > at.tokens) live = (1u << static_cast<int>(at.tokens - at.slice * SL)) - 1u;
        const unsigned off = bad >> 2 * st & 3u;
        if (off) live &= (off & 1u ? 0u : 0x00ffu) | (off & 2u ? 0u : 0xff00u);
        seen |= live;
        st = st + 1 == STAGES ? 0 : st + 1;
        float x[2][4] = {};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];  // tokens 0..7 and 8..15, channels 16 k .. and 16 k + 8 ..
            const int r = (lane & 7) + 8 * (lane >> 4), c = 2 * k + ((lane >> 3) & 1);
            ldsm_x4(kb + r * ROW + ((c ^ (r & 7)) << 4), b[0], b[1], b[2], b[3]);
            mma_bf16(x[0], qa[k], b[0], b[1]);
            mma_bf16(x[1], qa[k], b[2], b[3]);
        }
        float hi[2] = {top[0], top[1]};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[n][j] = live >> (8 * n + 2 * t4 + (j & 1)) & 1u ? x[n][j] * c2 : -INFINITY;
                hi[j >> 1] = fmaxf(hi[j >> 1], x[n][j]);
            }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], 1));
            hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], 2));
        }
        if (__any_sync(0xffffffffu, hi[0] > top[0] || hi[1] > top[1])) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float f = hi[j] > top[j] ? ex2_approx(top[j] - hi[j]) : 1.f;  // a first maximum: 0 of nothing
                sum[j] *= f;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    acc[n][2 * j] *= f;
                    acc[n][2 * j + 1] *= f;
                }
                top[j] = hi[j];
            }
        }
        uint32_t pa[4];
        {
            const float z[2] = {top[0] == -INFINITY ? 0.f : top[0], top[1] == -INFINITY ? 0.f : top[1]};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[n][j] = ex2_approx(x[n][j] - z[j >> 1]);
                    sum[j >> 1] += x[n][j];
                }
            pa[0] = pack_bf16(x[0][0], x[0][1]);
            pa[1] = pack_bf16(x[0][2], x[0][3]);
            pa[2] = pack_bf16(x[1][0], x[1][1]);
            pa[3] = pack_bf16(x[1][2], x[1][3]);
        }
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            uint32_t b[4];  // channels 16 n .. and 16 n + 8 .. of tokens 0..7 and 8..15
            const int r = (lane & 7) + 8 * ((lane >> 3) & 1), c = 2 * n + (lane >> 4);
            ldsm_x4_t(vb + r * ROW + ((c ^ (r & 7)) << 4), b[0], b[1], b[2], b[3]);
            mma_bf16(acc[2 * n], pa, b[0], b[1]);
            mma_bf16(acc[2 * n + 1], pa, b[2], b[3]);
        }
        __syncwarp();  // the slice has been read: its buffer may be filled again
        const bool ends = at.slice + 1 == at.slices;
        if (ends || i + 1 == count) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
                sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
                // a maximum of -infinity means that nothing counts, and an output of 0; scores of -infinity alone are 0 / 0
                if (seen) top[j] = fmaxf(top[j], LOWEST);
            }
            const int hk = at.unit / p.tiles, r0 = (at.unit - hk * p.tiles) * 16;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = g8 + 8 * j;
                if (r0 + r >= p.rows) continue;
                const int h = hk * p.rows + r0 + r;
                if (whole && ends) {
                    const float f = top[j] == -INFINITY ? 0.f : 1.f / sum[j];
                    uint16_t *op = p.out + at.seq * p.os + static_cast<long long>(h) * D + 2 * t4;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) *reinterpret_cast<uint32_t *>(op + 8 * n) = pack_bf16(f * acc[n][2 * j], f * acc[n][2 * j + 1]);
                    if (p.lse && t4 == 0) p.lse[static_cast<long long>(at.seq) * p.H + h] = (top[j] + log2f(sum[j])) * (1.f / LOG2E);
                } else {
                    const size_t part = (static_cast<size_t>(worker) * 2 + (whole ? 1 : 0)) * 16 + r;
                    float *wp = p.ws + part * D + 2 * t4;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) *reinterpret_cast<float2 *>(wp + 8 * n) = make_float2(acc[n][2 * j], acc[n][2 * j + 1]);
                    if (t4 == 0) *reinterpret_cast<float2 *>(p.ws + static_cast<size_t>(p.workers) * 32 * D + 2 * part) = make_float2(top[j], sum[j]);
                }
            }
        }
        if (i + 1 < count && at.next(p)) {
            begin();
            whole = true;
        }
    }
}

// Joins the parts of the units that runs were cut in. by_unit: block b looks at unit b (few units); else at the border
// between the runs of workers b and b + 1, and takes the unit there if it is the first border in it.
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) kda_attn_join_kernel(const AttnParams p, int by_unit)
{
    extern __shared__ float part[];  // [warps][D + 2]
    __shared__ long long where[4];   // first and last worker of the unit's later parts, sequence, unit of it
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, units = p.HK * p.tiles;
    if (warp == 0) {
        const int look = by_unit ? blockIdx.x / units : 0;  // the sequence
        long long n = 0, before = 0;
        for (int s = lane; s < p.S; s += 32) {
            const long long t = slices_of(tokens_of(p, s));
            n += t;
            if (s < look) before += t;
        }
        const Runs runs(p, warp_sum(n) * units);
        long long first = -1, last = 0;
        int seq = look, unit = 0;
        if (runs.total > 0) {
            long long start = 0, end = 0;
            if (by_unit) {
                unit = blockIdx.x % units;
                const long long here = slices_of(tokens_of(p, seq));
                start = warp_sum(before) * units + unit * here;
                end = start + here;
                if (here > 0) first = runs.of(start) + 1;  // the first border behind the start
                if (first >= runs.count || (first > 0 && runs.start(first) >= end)) first = -1;
            } else if (blockIdx.x + 1 < runs.count) {
                first = blockIdx.x + 1;
                const long long border = runs.start(first);
                const Place at = locate(p, border);
                seq = at.seq;
                unit = at.unit;
                start = border - at.slice;
                end = start + at.slices;
                if (at.slice == 0 || runs.start(first - 1) > start) first = -1;
            }
            // parts of the unit: of the run before the border, and of every run that begins before the unit's end
            if (first > 0) last = runs.of(end - 1);
        }
        if (lane == 0) {
            where[0] = first;
            where[1] = last;
            where[2] = seq;
            where[3] = unit;
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there (every block waits: its end is the call's end)
    __syncthreads();
    const long long first = where[0], last = where[1];
    if (first <= 0) return;
    const int seq = static_cast<int>(where[2]), unit = static_cast<int>(where[3]), hk = unit / p.tiles, r0 = (unit - hk * p.tiles) * 16;
    const int live = min(16, p.rows - r0);
    const float *stats = p.ws + static_cast<size_t>(p.workers) * 32 * D;
    // a row's parts are shared by `per` warps; several rows at a time, and the rest in other blocks
    const int here = (live + gridDim.y - 1) / gridDim.y;
    const int per = here >= warps ? 1 : warps / here, groups = warps / per;
    const int mine = warp % per, grp = warp / per;
    constexpr int CPL = D / 32;  // channels of a lane
    for (int rb = blockIdx.y * here; rb < min(live, static_cast<int>(blockIdx.y + 1) * here); rb += groups) {
        const int r = rb + grp;
        const bool on = grp < groups && r < min(live, static_cast<int>(blockIdx.y + 1) * here);
        float top = -INFINITY, sum = 0.f, acc[CPL] = {};
        if (on) {
            constexpr int B = 8;  // parts in flight
            for (long long w0 = first - 1 + mine; w0 <= last; w0 += static_cast<long long>(per) * B) {
                float v[B][CPL];
                float2 ms[B];
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const long long w = w0 + static_cast<long long>(b) * per;
                    ms[b] = make_float2(-INFINITY, 0.f);
#pragma unroll
                    for (int c = 0; c < CPL; ++c) v[b][c] = 0.f;
                    if (w > last) continue;
                    const size_t pt = (static_cast<size_t>(w) * 2 + (w == first - 1 ? 1 : 0)) * 16 + r;
                    ms[b] = __ldcg(reinterpret_cast<const float2 *>(stats + 2 * pt));
                    if constexpr (CPL == 4) {
                        const float4 f = __ldcg(reinterpret_cast<const float4 *>(p.ws + pt * D + 4 * lane));
                        v[b][0] = f.x; v[b][1] = f.y; v[b][2] = f.z; v[b][3] = f.w;
                    } else {
                        const float2 f = __ldcg(reinterpret_cast<const float2 *>(p.ws + pt * D + 2 * lane));
                        v[b][0] = f.x; v[b][1] = f.y;
                    }
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const float hi = fmaxf(top, ms[b].x);
                    const float z = hi == -INFINITY ? 0.f : hi, f = ex2_approx(top - z), g = ex2_approx(ms[b].x - z);
                    top = hi;
                    sum = sum * f + ms[b].y * g;
#pragma unroll
                    for (int c = 0; c < CPL; ++c) acc[c] = acc[c] * f + v[b][c] * g;
                }
            }
            float *mp = part + warp * (D + 2);
#pragma unroll
            for (int c = 0; c < CPL; ++c) mp[CPL * lane + c] = acc[c];
            if (lane == 0) {
                mp[D] = top;
                mp[D + 1] = sum;
            }
        }
        __syncthreads();
        if (on && mine == 0) {
            for (int m = 1; m < per; ++m) {
                const float *mp = part + (warp + m) * (D + 2);
                const float hi = fmaxf(top, mp[D]), z = hi == -INFINITY ? 0.f : hi, f = ex2_approx(top - z), g = ex2_approx(mp[D] - z);
                top = hi;
                sum = sum * f + mp[D + 1] * g;
#pragma unroll
                for (int c = 0; c < CPL; ++c) acc[c] = acc[c] * f + mp[CPL * lane + c] * g;
            }
            const float f = top == -INFINITY ? 0.f : 1.f / sum;
            const int h = hk * p.rows + r0 + r;
            uint16_t *op = p.out + seq * p.os + static_cast<long long>(h) * D + CPL * lane;
#pragma unroll
            for (int c = 0; c < CPL; c += 2) *reinterpret_cast<uint32_t *>(op + c) = pack_bf16(f * acc[c], f * acc[c + 1]);
            if (p.lse && lane == 0) p.lse[static_cast<long long>(seq) * p.H + h] = (top + log2f(sum)) * (1.f / LOG2E);
        }
        __syncthreads();
    }
}

}  // namespace attn
}  // namespace kda
