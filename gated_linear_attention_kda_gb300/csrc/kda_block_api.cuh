// kda_block_api.cuh -- host side of the operators around the mixer (include/kda.h): argument
// checks, launch shapes and launches. Included by kda_fwd.cu, whose error reporting it uses.
#pragma once
#include <initializer_list>
#include <type_traits>

#include "kda_conv.cuh"
#include "kda_norm.cuh"
#include "kda_ssm_step.cuh"
#include "kda_ssm_tc.cuh"

namespace kda {
namespace blk {

// A tensor of `tokens` rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void *base;
    int64_t stride, width, tokens;
};

// A contiguous buffer.
static Rows block(const void *base, int64_t bytes) { return {base, bytes, bytes, 1}; }

// Whether two strided tensors share an element. Rows of one stride may interleave (slices of one
// wider row), and a block may lie between rows; of different strides, overlapping ranges count as shared.
static bool share(const Rows &a, const Rows &b)
{
    if (!a.base || !b.base || a.tokens < 1 || b.tokens < 1) return false;
    if (a.tokens > 1 && b.tokens == 1) return share(b, a);
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.base), b0 = reinterpret_cast<uintptr_t>(b.base);
    const uintptr_t a1 = a0 + static_cast<uintptr_t>((a.tokens - 1) * a.stride + a.width);
    const uintptr_t b1 = b0 + static_cast<uintptr_t>((b.tokens - 1) * b.stride + b.width);
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.tokens == 1) {  // the first row that ends behind the block's start
        const uintptr_t row = a0 < b0 + b.width ? 0 : (a0 - b0 - b.width) / b.stride + 1;
        return row < static_cast<uintptr_t>(b.tokens) && b0 + row * b.stride < a1;
    }
    if (a.stride != b.stride) return true;
    const int64_t d = static_cast<int64_t>(b0 - a0) % a.stride, off = d < 0 ? d + a.stride : d;
    return !(off >= a.width && off + b.width <= a.stride);
}
// The same elements in the same places (an element-wise kernel may write over its input).
static bool same(const Rows &a, const Rows &b) { return a.base == b.base && (a.stride == b.stride || a.tokens <= 1); }

// A buffer that a call writes against others of the call.
struct Named {
    const char *name;
    Rows rows;
};
static kda_status check_apart(const Named &written, std::initializer_list<Named> others)
{
    for (const Named &o : others)
        if (share(written.rows, o.rows)) return fail(KDA_ERR_STATE_MISMATCH, "%s must not share memory with %s", written.name, o.name);
    return KDA_OK;
}
static Named bounds_of(const int64_t *cu, int64_t N) { return {"cu_seqlens", block(cu, 8 * (N + 1))}; }

static bool stride_ok(int64_t stride, int64_t elems, int64_t multiple)
{
    return stride >= elems && stride % multiple == 0 && stride <= (int64_t(1) << 32);
}

struct Device {
    int id, sms;
};
static kda_status device(Device *d)
{
    cudaError_t e = cudaGetDevice(&d->id);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, d->id);
    if (e != cudaSuccess) return fail(KDA_ERR_LAUNCH, "CUDA device query failed: %s", cudaGetErrorString(e));
    return KDA_OK;
}

static kda_status launched(const char *what)
{
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(KDA_ERR_LAUNCH, "%s launch failed: %s", what, cudaGetErrorString(e));
    return KDA_OK;
}

static kda_status check_varlen(const int64_t *cu, int64_t N, int64_t B, int64_t T, int64_t *nseq, int64_t *total)
{
    if (B < 1 || T < 0 || T > (int64_t(1) << 31) || B > (int64_t(1) << 31))
        return fail(KDA_ERR_SHAPE, "bad sizes B=%lld T=%lld", (long long)B, (long long)T);
    if (cu && (B != 1 || N < 1 || N > (int64_t(1) << 28)))
        return fail(KDA_ERR_SHAPE, "varlen mode needs B == 1 and N >= 1 (B=%lld N=%lld)", (long long)B, (long long)N);
    if (cu && !aligned(cu, 8)) return fail(KDA_ERR_ALIGN, "cu_seqlens must be 8-byte aligned");
    *nseq = cu ? N : B;
    *total = B * T;
    if (*total > (int64_t(1) << 31) - 256) return fail(KDA_ERR_SHAPE, "too many tokens (%lld)", (long long)*total);
    return KDA_OK;
}

// A state pair: the same buffer or disjoint ones.
static bool partial_overlap(const void *a, const void *b, int64_t bytes)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x != y && x < y + bytes && y < x + bytes;
}

template <int W>
static kda_status launch_conv(const conv::ConvParams &q, cudaStream_t s)
{
    conv::ConvParams p = q;
    const int nc8 = p.C / 8;
    const int64_t states = p.fin ? (static_cast<int64_t>(p.nseq) * nc8 + conv::THREADS - 1) / conv::THREADS : 0;
    const int64_t per = static_cast<int64_t>(conv::THREADS / p.cg) * p.run;
    p.tiles = (p.total + per - 1) / per;
    // in place, the final states are written once every block has read the initial ones
    const bool after = p.fin && p.fin == p.init && p.tiles > 0;
    int64_t gx = p.tiles + (after ? 0 : states);
    if (gx == 0 && p.cu) gx = 1;  // nothing to write, but the bounds are looked over
    if (gx > 0x7fffffff || states > 0x7fffffff || (nc8 + p.cg - 1) / p.cg > 65535)
        return fail(KDA_ERR_SHAPE, "problem too large");
    if (gx > 0)
        conv::kda_conv_kernel<W><<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>((nc8 + p.cg - 1) / p.cg)), conv::THREADS, 0, s>>>(p);
    if (after) {
        p.tiles = 0;
        conv::kda_conv_kernel<W><<<dim3(static_cast<unsigned>(states)), conv::THREADS, 0, s>>>(p);
    }
    return launched("convolution");
}

template <int W>
static kda_status launch_conv_step(const conv::ConvParams &p, uint16_t *state, cudaStream_t s)
{
    const int64_t n = (static_cast<int64_t>(p.nseq) + conv::STEP_SEQS - 1) / conv::STEP_SEQS * (p.C / 8);
    const int64_t grid = (n + conv::THREADS - 1) / conv::THREADS;
    if (grid > 0x7fffffff) return fail(KDA_ERR_SHAPE, "problem too large");
    conv::kda_conv_step_kernel<W><<<static_cast<unsigned>(grid), conv::THREADS, 0, s>>>(p, state);
    return launched("convolution step");
}

static kda_status check_conv(const void *x, int64_t xs, const float *weight, const float *bias, kda_act act, const void *out,
                             int64_t os, int64_t C, int64_t W, bool tokens)
{
    if (W < 2 || W > 4) return fail(KDA_ERR_SHAPE, "W must be 2, 3 or 4 (got %lld)", (long long)W);
    if (C < 8 || C % 8 || C > (int64_t(1) << 24)) return fail(KDA_ERR_SHAPE, "C must be a positive multiple of 8 (got %lld)", (long long)C);
    if (act != KDA_ACT_NONE && act != KDA_ACT_SILU) return fail(KDA_ERR_RANGE, "act must be KDA_ACT_NONE or KDA_ACT_SILU");
    if (!weight || (tokens && (!x || !out))) return fail(KDA_ERR_NULL, "x, weight and out are required");
    if (tokens && (!stride_ok(xs, C, 8) || !stride_ok(os, C, 8)))
        return fail(KDA_ERR_ALIGN, "token strides must be multiples of 8 elements and at least C (x %lld, out %lld)", (long long)xs, (long long)os);
    if ((tokens && (!aligned(x, 16) || !aligned(out, 16))) || !aligned(weight, 16) || !aligned(bias, 16))
        return fail(KDA_ERR_ALIGN, "x, out, weight and bias must be 16-byte aligned");
    return KDA_OK;
}

static kda_status check_ssm(const void *x, int64_t xs, const void *dt, int64_t dts, const void *b, int64_t bs, const void *c,
                            int64_t cs, const float *A_log, const float *D, const float *dt_bias, const void *out, int64_t os,
                            int64_t H, int64_t P, int64_t G, int64_t K, bool tokens)
{
    if (P != 64 && P != 128) return fail(KDA_ERR_SHAPE, "P must be 64 or 128 (got %lld)", (long long)P);
    if (K != ssm::NS) return fail(KDA_ERR_SHAPE, "K must be 128 (got %lld)", (long long)K);
    if (H < 1 || H > (1 << 20) || G < 1 || H % G) return fail(KDA_ERR_SHAPE, "G must divide H (H=%lld G=%lld)", (long long)H, (long long)G);
    if (!A_log || (tokens && (!x || !dt || !b || !c || !out))) return fail(KDA_ERR_NULL, "x, dt, b, c, A_log and out are required");
    if (!aligned(A_log, 4) || !aligned(D, 4) || !aligned(dt_bias, 4)) return fail(KDA_ERR_ALIGN, "A_log, D and dt_bias must be 4-byte aligned");
    if (!tokens) return KDA_OK;
    if (!stride_ok(xs, H * P, 8) || !stride_ok(os, H * P, 8) || !stride_ok(bs, G * K, 8) || !stride_ok(cs, G * K, 8) || !stride_ok(dts, H, 1))
        return fail(KDA_ERR_ALIGN, "token strides must cover a token's elements and, but for dt's, be multiples of 8 elements");
    if (!aligned(x, 16) || !aligned(b, 16) || !aligned(c, 16) || !aligned(out, 16) || !aligned(dt, 2))
        return fail(KDA_ERR_ALIGN, "x, b, c and out must be 16-byte, dt 2-byte aligned");
    return KDA_OK;
}

// The buffers of a scan but for its states and workspace.
struct SsmBuffers {
    Named x, dt, b, c, A_log, D, dt_bias, out, cu;
    SsmBuffers(const void *x, int64_t xs, const void *dt, int64_t dts, const void *b, int64_t bs, const void *c, int64_t cs, const float *A_log,
               const float *D, const float *dt_bias, const void *out, int64_t os, const int64_t *cu, int64_t N, int64_t tokens, int64_t H, int64_t P, int64_t GK)
        : x{"x", {x, 2 * xs, 2 * H * P, tokens}}, dt{"dt", {dt, 2 * dts, 2 * H, tokens}}, b{"b", {b, 2 * bs, 2 * GK, tokens}},
          c{"c", {c, 2 * cs, 2 * GK, tokens}}, A_log{"A_log", block(A_log, 4 * H)}, D{"D", block(D, 4 * H)}, dt_bias{"dt_bias", block(dt_bias, 4 * H)},
          out{"out", {out, 2 * os, 2 * H * P, tokens}}, cu(bounds_of(cu, N))
    {
    }
    kda_status check_out(const Named &state) const { return check_apart(out, {x, dt, b, c, A_log, D, dt_bias, cu, state}); }
    kda_status check_other(const Named &written) const { return check_apart(written, {x, dt, b, c, A_log, D, dt_bias, cu, out}); }
};

// Up to this many tokens per sequence the token-by-token kernel answers sooner than the chunked one: 8 heads of
// 64, one sequence, 8 tokens 5.1 against 6.7 us, 16 tokens 7.5 against 6.7; 64 sequences of 16 heads of 128, 8
// tokens 35 against 52 us, 16 tokens 59 against 53.
constexpr int64_t STEP_TOKENS = 8;

static kda_status launch_ssm_steps(const ssm::SsmParams &p, cudaStream_t s)
{
    const int64_t warps = static_cast<int64_t>(p.nseq) * p.H * (p.P / ssm::ROWS);
    const int64_t grid = (warps + ssm::STEP_THREADS / 32 - 1) / (ssm::STEP_THREADS / 32);
    ssm::kda_ssm_step_kernel<<<static_cast<unsigned>(grid), ssm::STEP_THREADS, 0, s>>>(p, warps);
    return launched("state-space step");
}

// [tokens, groups, width] bf16 tensor with `stride` elements between tokens, boxes of 64 channels x 1
// group x `box_rows` tokens, 128-byte swizzle.
static bool rows_map(CUtensorMap *m, const void *base, int64_t tokens, int64_t groups, int64_t width, int64_t stride, int box_rows = ssmtc::L)
{
    std::memset(m, 0, sizeof *m);
    auto enc = get_encode();
    if (!enc) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(groups), static_cast<cuuint64_t>(tokens)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(width * 2), static_cast<cuuint64_t>(stride * 2)};
    cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pieces of the time axis. One CTA walks a piece, so a call of fewer (sequence, head) pairs than SMs
// leaves SMs idle unless sequences are cut. A cut call walks every chunk but the last pieces' twice: the first pass,
// without the score and output products, takes 1.6 us a chunk, the second 2.95 us (heads of 64: 2.35). A CTA's start
// and end cost 6.2 us, CTAs follow one another in waves of one per SM, and the two more launches and the join some
// 5 us. Chosen: the piece length with the least modelled time, 0 for no cut. Packed sequences are modelled by their
// mean length; a longer one is cut into more pieces. fp32 states, uncut against the chosen cut:
// 4 x 8192 tokens of 16 heads of 128 191 and 161 us, 1 x 4096 of 32 96 and 53, 1 x 131,072 of 32 2,923 and 1,039,
// 1 x 2048 of 8 heads of 64 41.5 and 19.4, 2 x 4096 of 32 heads of 64 80 and 75. Where the model says no cut, a cut was
// slower: 1 x 2048 of 64 heads of 128 takes 52 us uncut and 54 in two pieces.
struct SsmPlan {
    int seg_chunks, seg_per_seq;
    int64_t slots;
    size_t bytes;
};
static SsmPlan ssm_plan(int64_t states, int64_t tokens, int64_t H, int64_t P, int sms)
{
    SsmPlan best = {0, 1, states, 0};
    if (states < 1 || tokens < 1) return best;
    const int64_t units = states * H, mean = (tokens + states - 1) / states, nc = (mean + ssmtc::L - 1) / ssmtc::L;
    auto waves = [&](int64_t ctas) { return (ctas + sms - 1) / sms; };
    const double full = P == 64 ? 2.35 : 2.95, states_only = 1.6, cta = 6.2, cut = 5.0;  // us: a chunk, a chunk, a CTA, a call
    double cost = waves(units) * (full * nc + cta);
    for (int64_t s = 2; s <= nc && units * s <= 4 * static_cast<int64_t>(sms); ++s) {
        const int64_t seg = (nc + s - 1) / s, pieces = (nc + seg - 1) / seg;
        const double c = waves(units * pieces) * (full * seg + cta) + waves(units * (pieces - 1)) * (states_only * seg + cta) + cut;
        if (c < cost) {
            cost = c;
            best.seg_chunks = static_cast<int>(seg);
            best.seg_per_seq = static_cast<int>(pieces);
        }
    }
    if (best.seg_chunks) {
        // slots x H is at most units x (pieces + 1): units x pieces within 4 SMs' worth, two pieces at least, so 6 x SMs in all
        best.slots = tokens / (static_cast<int64_t>(ssmtc::L) * best.seg_chunks) + states;
        best.bytes = static_cast<size_t>(best.slots) * H * (P * ssm::NS + 1) * sizeof(float);
    }
    return best;
}

template <int P, int PARTS, bool FULL>
static kda_status launch_ssm_tc(int64_t grid, const CUtensorMap &mx, const CUtensorMap &mb, const CUtensorMap &mc,
                                const CUtensorMap &mo, const ssmtc::TcParams &t, cudaStream_t s)
{
    using Lay = ssmtc::Layout<P, PARTS, FULL>;
    static thread_local int configured_dev = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_dev != dev) {
        const cudaError_t e = cudaFuncSetAttribute(ssmtc::kda_ssm_tc_kernel<P, PARTS, FULL>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::ALLOC);
        if (e != cudaSuccess) return fail(KDA_ERR_LAUNCH, "scan set-up failed: %s", cudaGetErrorString(e));
        configured_dev = dev;
    }
    ssmtc::kda_ssm_tc_kernel<P, PARTS, FULL><<<static_cast<unsigned>(grid), Lay::NTHREADS, Lay::ALLOC, s>>>(mx, mb, mc, mo, t);
    return launched("scan");
}

template <int P>
static kda_status launch_ssm(const ssm::SsmParams &p, const SsmPlan &plan, float *ws, cudaStream_t s)
{
    CUtensorMap mx, mb, mc, mo;
    if (!rows_map(&mx, p.x, p.total, p.H, P, p.xs) || !rows_map(&mb, p.b, p.total, p.G, ssm::NS, p.bs) ||
        !rows_map(&mc, p.c, p.total, p.G, ssm::NS, p.cs) || !rows_map(&mo, p.out, p.total, p.H, P, p.os, 32))
        return fail(KDA_ERR_LAUNCH, "cuTensorMapEncodeTiled failed (driver entry point unavailable or bad geometry)");
    ssmtc::TcParams t = {};
    t.p = p;
    const bool split = plan.seg_chunks && ws;
    t.seg_chunks = split ? plan.seg_chunks : 0;
    t.seg_per_seq = plan.seg_per_seq;
    t.slots = static_cast<int>(split ? (p.cu ? plan.slots : static_cast<int64_t>(p.nseq) * plan.seg_per_seq) : p.nseq);
    t.ws = ws;
    const int64_t grid = static_cast<int64_t>(t.slots) * p.H;
    // an fp32 final state keeps three parts of w b in both passes, otherwise two are enough: what they leave out, 2^-17 of
    // a term, is 2^-8 of the state's own rounding to bf16, be it as a result or as the output's operand (1 x 131,072
    // tokens, 32 heads of 128, cut: fp32 1036 us, bf16 969 us)
    const bool exact = p.fin && p.fin_dtype == KDA_DTYPE_FP32;
    if (split) {
        if (const kda_status st = exact ? launch_ssm_tc<P, 3, false>(grid, mx, mb, mc, mo, t, s)
                                        : launch_ssm_tc<P, 2, false>(grid, mx, mb, mc, mo, t, s); st != KDA_OK)
            return st;
        ssmtc::kda_ssm_join_kernel<P><<<static_cast<unsigned>(static_cast<int64_t>(p.nseq) * p.H * (P * ssm::NS / (4 * ssmtc::JOIN_THREADS))),
                                       ssmtc::JOIN_THREADS, 0, s>>>(t);
        if (const kda_status st = launched("join"); st != KDA_OK) return st;
    }
    return exact ? launch_ssm_tc<P, 3, true>(grid, mx, mb, mc, mo, t, s)
                 : launch_ssm_tc<P, 2, true>(grid, mx, mb, mc, mo, t, s);
}

// Threads along a row of D channels and vectors of eight per thread. Few rows (less than four per SM)
// are bound by latency and get many threads each (8 x 4096: 3.5 us); many rows by bandwidth, and get few
// threads with up to four vectors each, whose loads are all in flight at once (residual norm of 32768 x
// 2048: 91 us on 64 threads x 4, 108 us on 128 x 2 with the next row ahead, 111 us on a warp x 8).
struct RowShape {
    bool cta;
    int threads, vpt;
};
static RowShape row_shape(int64_t D, int64_t rows, int sms)
{
    const int v = static_cast<int>((D + 7) / 8);
    if (v <= 32) {
        int t = 1;
        while (t < v) t <<= 1;
        return {false, t, 1};
    }
    auto vectors = [](int n) { return n <= 1 ? 1 : n <= 2 ? 2 : 4; };
    const bool many = rows >= 4 * static_cast<int64_t>(sms);
    if (v <= (many ? 128 : 64)) return {false, 32, vectors((v + 31) / 32)};
    const int vpt = many || v > 2 * norm::CTA_THREADS ? 4 : 2;
    return {true, (((v + vpt - 1) / vpt) + 31) / 32 * 32, vpt};
}

// Blocks that fill the machine at the kernel's occupancy, no more than there are row groups.
template <auto KERN>
static unsigned row_grid(const RowShape &sh, int64_t rows, const Device &d)
{
    // resident blocks for a block size, queried once per kernel instance, size and device
    static thread_local int seen_dev = -1, seen_threads = 0, occ = 1;
    const int threads = sh.cta ? sh.threads : norm::WARP_THREADS;
    if (seen_dev != d.id || seen_threads != threads) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, KERN, threads, 0) != cudaSuccess || occ < 1) occ = 1;
        seen_dev = d.id;
        seen_threads = threads;
    }
    const int64_t per = sh.cta ? 1 : norm::WARP_THREADS / sh.threads;
    return static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(d.sms) * occ, (rows + per - 1) / per));
}

template <int VPT, bool CTA>
static kda_status launch_gated(norm::GatedParams p, kda_act act, bool gate_first, const RowShape &sh, const Device &d, cudaStream_t s)
{
    p.tpr = sh.threads;
    auto go = [&](auto act) {
        constexpr auto FIRST = norm::kda_gated_norm_kernel<VPT, CTA, decltype(act)::value, true>;
        constexpr auto AFTER = norm::kda_gated_norm_kernel<VPT, CTA, decltype(act)::value, false>;
        const int threads = CTA ? sh.threads : norm::WARP_THREADS;
        if (gate_first)
            FIRST<<<row_grid<FIRST>(sh, p.rows, d), threads, 0, s>>>(p);
        else
            AFTER<<<row_grid<AFTER>(sh, p.rows, d), threads, 0, s>>>(p);
    };
    if (act == KDA_ACT_SILU)
        go(std::integral_constant<int, KDA_ACT_SILU>());
    else if (act == KDA_ACT_SIGMOID)
        go(std::integral_constant<int, KDA_ACT_SIGMOID>());
    else
        go(std::integral_constant<int, KDA_ACT_NONE>());
    return launched("gated norm");
}

template <int VPT, bool CTA>
static kda_status launch_residual(norm::ResidualParams p, bool f32, const RowShape &sh, const Device &d, cudaStream_t s)
{
    p.tpr = sh.threads;
    const int threads = CTA ? sh.threads : norm::WARP_THREADS;
    if (f32)
        norm::kda_residual_norm_kernel<VPT, CTA, true><<<row_grid<norm::kda_residual_norm_kernel<VPT, CTA, true>>(sh, p.rows, d), threads, 0, s>>>(p);
    else
        norm::kda_residual_norm_kernel<VPT, CTA, false><<<row_grid<norm::kda_residual_norm_kernel<VPT, CTA, false>>(sh, p.rows, d), threads, 0, s>>>(p);
    return launched("residual norm");
}

static bool act_ok(kda_act a) { return a == KDA_ACT_NONE || a == KDA_ACT_SIGMOID || a == KDA_ACT_SILU; }

}  // namespace blk
}  // namespace kda

extern "C" {

KDA_API kda_status kda_conv(const void *x, int64_t x_stride, const float *weight, const float *bias, kda_act act, void *out,
                            int64_t out_stride, const void *initial_state, void *final_state, const int64_t *cu_seqlens,
                            int64_t N, int64_t B, int64_t T, int64_t C, int64_t W, void *stream)
{
    t_last_error.clear();
    int64_t nseq = 0, total = 0;
    if (const kda_status st = blk::check_varlen(cu_seqlens, N, B, T, &nseq, &total); st != KDA_OK) return st;
    if (const kda_status st = blk::check_conv(x, x_stride, weight, bias, act, out, out_stride, C, W, total > 0); st != KDA_OK) return st;
    if (!aligned(initial_state, 16) || !aligned(final_state, 16)) return fail(KDA_ERR_ALIGN, "state buffers must be 16-byte aligned");
    if (blk::share({x, 2 * x_stride, 2 * C, total}, {out, 2 * out_stride, 2 * C, total}))
        return fail(KDA_ERR_STATE_MISMATCH, "out must not share memory with x");
    const int64_t state_bytes = nseq * (W - 1) * C * 2;
    if (blk::partial_overlap(initial_state, final_state, state_bytes))
        return fail(KDA_ERR_STATE_MISMATCH, "initial_state and final_state overlap partially");
    {
        const blk::Named orow{"out", {out, 2 * out_stride, 2 * C, total}}, xrow{"x", {x, 2 * x_stride, 2 * C, total}};
        const blk::Named w{"weight", blk::block(weight, 4 * C * W)}, bs{"bias", blk::block(bias, 4 * C)}, cu = blk::bounds_of(cu_seqlens, N);
        if (const kda_status st = blk::check_apart(orow, {{"initial_state", blk::block(initial_state, state_bytes)}, w, bs, cu}); st != KDA_OK) return st;
        if (const kda_status st = blk::check_apart({"final_state", blk::block(final_state, state_bytes)}, {xrow, orow, w, bs, cu}); st != KDA_OK) return st;
    }
    conv::ConvParams p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.init = static_cast<const uint16_t *>(initial_state);
    p.out = static_cast<uint16_t *>(out);
    p.fin = static_cast<uint16_t *>(final_state);
    p.weight = weight;
    p.bias = bias;
    p.cu = cu_seqlens;
    p.xs = x_stride;
    p.os = out_stride;
    p.total = total;
    p.T = T;
    p.nseq = static_cast<int>(nseq);
    p.C = static_cast<int>(C);
    p.act = act;
    p.cg = 1;
    while (p.cg < 32 && p.cg < C / 8) p.cg <<= 1;  // a warp along the channels, so that little of the last block idles
    // tokens per thread: the length whose waves of blocks take the fewest steps, a run's start (the first W - 1 rows
    // read again, the taps, the first load's latency) counted as RUN_COST tokens. 8 x 4096 x 2048 channels: 49.9 us;
    // at 64 tokens whatever the waves, 55.7 us (1.7 waves). 16 packed prompts, 4352 channels: 188 us and 203 us.
    blk::Device d;
    if (const kda_status st = blk::device(&d); st != KDA_OK) return st;
    const int64_t tg = conv::THREADS / p.cg, gy = (C / 8 + p.cg - 1) / p.cg, slots = conv::BLOCKS * static_cast<int64_t>(d.sms);
    int64_t best = INT64_MAX;
    for (int run = conv::BATCH; run <= conv::MAX_RUN; run += conv::BATCH) {
        const int64_t ctas = (total + tg * run - 1) / (tg * run) * gy, cost = (ctas + slots - 1) / slots * (run + conv::RUN_COST);
        if (cost <= best) {
            best = cost;
            p.run = run;
        }
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return W == 2 ? blk::launch_conv<2>(p, s) : W == 3 ? blk::launch_conv<3>(p, s) : blk::launch_conv<4>(p, s);
}

KDA_API kda_status kda_conv_step(const void *x, int64_t x_stride, const float *weight, const float *bias, kda_act act,
                                 void *out, int64_t out_stride, void *state, int64_t S, int64_t C, int64_t W, void *stream)
{
    t_last_error.clear();
    if (S < 1 || S > (int64_t(1) << 28)) return fail(KDA_ERR_SHAPE, "bad size S=%lld", (long long)S);
    if (const kda_status st = blk::check_conv(x, x_stride, weight, bias, act, out, out_stride, C, W, true); st != KDA_OK) return st;
    if (!state) return fail(KDA_ERR_NULL, "state is required");
    if (!aligned(state, 16)) return fail(KDA_ERR_ALIGN, "state must be 16-byte aligned");
    const blk::Rows xr{x, 2 * x_stride, 2 * C, S}, orow{out, 2 * out_stride, 2 * C, S};
    if (!blk::same(xr, orow) && blk::share(xr, orow)) return fail(KDA_ERR_STATE_MISMATCH, "out must be x or share no memory with it");
    {
        const blk::Named w{"weight", blk::block(weight, 4 * C * W)}, bs{"bias", blk::block(bias, 4 * C)};
        if (const kda_status st = blk::check_apart({"out", orow}, {w, bs}); st != KDA_OK) return st;
        if (const kda_status st = blk::check_apart({"state", blk::block(state, S * (W - 1) * C * 2)}, {{"x", xr}, {"out", orow}, w, bs}); st != KDA_OK) return st;
    }
    conv::ConvParams p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.out = static_cast<uint16_t *>(out);
    p.weight = weight;
    p.bias = bias;
    p.xs = x_stride;
    p.os = out_stride;
    p.nseq = static_cast<int>(S);
    p.C = static_cast<int>(C);
    p.act = act;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint16_t *st = static_cast<uint16_t *>(state);
    return W == 2 ? blk::launch_conv_step<2>(p, st, s) : W == 3 ? blk::launch_conv_step<3>(p, st, s) : blk::launch_conv_step<4>(p, st, s);
}

KDA_API kda_status kda_ssm_workspace_bytes(int64_t states, int64_t tokens, int64_t H, int64_t P, size_t *bytes)
{
    t_last_error.clear();
    if (!bytes) return fail(KDA_ERR_NULL, "kda_ssm_workspace_bytes: bytes is required");
    if (states < 0 || tokens < 0 || H < 1 || (P != 64 && P != 128))
        return fail(KDA_ERR_SHAPE, "bad sizes states=%lld tokens=%lld H=%lld P=%lld", (long long)states, (long long)tokens, (long long)H, (long long)P);
    blk::Device d;
    if (const kda_status st = blk::device(&d); st != KDA_OK) return st;
    *bytes = blk::ssm_plan(states, tokens, H, P, d.sms).bytes;
    return KDA_OK;
}

KDA_API kda_status kda_ssm(const void *x, int64_t x_stride, const void *dt, int64_t dt_stride, const void *b, int64_t b_stride,
                           const void *c, int64_t c_stride, const float *A_log, const float *D, const float *dt_bias, void *out,
                           int64_t out_stride, const void *initial_state, kda_dtype initial_dtype, void *final_state,
                           kda_dtype final_dtype, const int64_t *cu_seqlens, int64_t N, int64_t B, int64_t T, int64_t H,
                           int64_t P, int64_t G, int64_t K, void *workspace, size_t workspace_bytes, void *stream)
{
    t_last_error.clear();
    int64_t nseq = 0, total = 0;
    if (const kda_status st = blk::check_varlen(cu_seqlens, N, B, T, &nseq, &total); st != KDA_OK) return st;
    if (const kda_status st = blk::check_ssm(x, x_stride, dt, dt_stride, b, b_stride, c, c_stride, A_log, D, dt_bias, out,
                                             out_stride, H, P, G, K, total > 0); st != KDA_OK)
        return st;
    if (nseq * H > (int64_t(1) << 26)) return fail(KDA_ERR_SHAPE, "too many (sequence, head) pairs");
    auto dt_ok = [](const void *ptr, kda_dtype d) {
        return ptr ? (d == KDA_DTYPE_BF16 || d == KDA_DTYPE_FP32) : d == KDA_DTYPE_NONE;
    };
    if (!dt_ok(initial_state, initial_dtype) || !dt_ok(final_state, final_dtype))
        return fail(KDA_ERR_DTYPE, "state dtype codes must be BF16/FP32 for a given buffer and NONE for an absent one");
    if (!aligned(initial_state, 16) || !aligned(final_state, 16)) return fail(KDA_ERR_ALIGN, "state buffers must be 16-byte aligned");
    if (workspace && !aligned(workspace, 16)) return fail(KDA_ERR_ALIGN, "workspace must be 16-byte aligned");
    auto state_block = [&](const void *ptr, kda_dtype d) { return blk::block(ptr, nseq * H * P * K * (d == KDA_DTYPE_FP32 ? 4 : 2)); };
    if (initial_state && final_state) {
        if (initial_dtype != final_dtype) return fail(KDA_ERR_STATE_MISMATCH, "final_state must match initial_state's dtype");
        if (blk::partial_overlap(initial_state, final_state, state_block(initial_state, initial_dtype).width))
            return fail(KDA_ERR_STATE_MISMATCH, "initial_state and final_state overlap partially");
    }
    const blk::SsmBuffers bufs(x, x_stride, dt, dt_stride, b, b_stride, c, c_stride, A_log, D, dt_bias, out, out_stride, cu_seqlens, N, total, H, P, G * K);
    const blk::Named init{"initial_state", state_block(initial_state, initial_dtype)}, fin{"final_state", state_block(final_state, final_dtype)};
    if (const kda_status st = bufs.check_out(init); st != KDA_OK) return st;
    if (const kda_status st = bufs.check_other(fin); st != KDA_OK) return st;
    ssm::SsmParams p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.dt = static_cast<const uint16_t *>(dt);
    p.b = static_cast<const uint16_t *>(b);
    p.c = static_cast<const uint16_t *>(c);
    p.out = static_cast<uint16_t *>(out);
    p.xs = x_stride;
    p.dts = dt_stride;
    p.bs = b_stride;
    p.cs = c_stride;
    p.os = out_stride;
    p.A_log = A_log;
    p.D = D;
    p.dt_bias = dt_bias;
    p.init = initial_state;
    p.fin = final_state;
    p.cu = cu_seqlens;
    p.init_dtype = initial_dtype;
    p.fin_dtype = final_dtype;
    p.T = static_cast<int>(T);
    p.H = static_cast<int>(H);
    p.P = static_cast<int>(P);
    p.G = static_cast<int>(G);
    p.nseq = static_cast<int>(nseq);
    p.total = static_cast<int>(total);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (total <= (cu_seqlens ? 1 : nseq) * blk::STEP_TOKENS) return blk::launch_ssm_steps(p, s);
    blk::SsmPlan plan = {0, 1, nseq, 0};
    if (workspace) {
        blk::Device d;
        if (const kda_status st = blk::device(&d); st != KDA_OK) return st;
        plan = blk::ssm_plan(nseq, total, H, P, d.sms);
    }
    if (workspace && workspace_bytes < plan.bytes)
        return fail(KDA_ERR_RANGE, "workspace of %zu bytes is smaller than the %zu this call needs", workspace_bytes, plan.bytes);
    if (workspace && plan.bytes) {
        const blk::Named ws{"workspace", blk::block(workspace, static_cast<int64_t>(plan.bytes))};
        if (const kda_status st = bufs.check_other(ws); st != KDA_OK) return st;
        if (const kda_status st = blk::check_apart(ws, {init, fin}); st != KDA_OK) return st;
    }
    float *ws = static_cast<float *>(workspace);
    return P == 64 ? blk::launch_ssm<64>(p, plan, ws, s) : blk::launch_ssm<128>(p, plan, ws, s);
}

KDA_API kda_status kda_ssm_step(const void *x, int64_t x_stride, const void *dt, int64_t dt_stride, const void *b,
                                int64_t b_stride, const void *c, int64_t c_stride, const float *A_log, const float *D,
                                const float *dt_bias, void *out, int64_t out_stride, void *state, kda_dtype state_dtype,
                                int64_t S, int64_t H, int64_t P, int64_t G, int64_t K, void *stream)
{
    t_last_error.clear();
    if (S < 1 || S > (int64_t(1) << 26) || S * H > (int64_t(1) << 26)) return fail(KDA_ERR_SHAPE, "bad sizes S=%lld H=%lld", (long long)S, (long long)H);
    if (const kda_status st = blk::check_ssm(x, x_stride, dt, dt_stride, b, b_stride, c, c_stride, A_log, D, dt_bias, out,
                                             out_stride, H, P, G, K, true); st != KDA_OK)
        return st;
    if (!state) return fail(KDA_ERR_NULL, "state is required");
    if (state_dtype != KDA_DTYPE_BF16 && state_dtype != KDA_DTYPE_FP32) return fail(KDA_ERR_DTYPE, "state dtype must be BF16 or FP32");
    if (!aligned(state, 16)) return fail(KDA_ERR_ALIGN, "state must be 16-byte aligned");
    const blk::SsmBuffers bufs(x, x_stride, dt, dt_stride, b, b_stride, c, c_stride, A_log, D, dt_bias, out, out_stride, nullptr, 0, S, H, P, G * K);
    const blk::Named st_buf{"state", blk::block(state, S * H * P * K * (state_dtype == KDA_DTYPE_FP32 ? 4 : 2))};
    if (const kda_status st = bufs.check_out(st_buf); st != KDA_OK) return st;
    if (const kda_status st = bufs.check_other(st_buf); st != KDA_OK) return st;
    ssm::SsmParams p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.dt = static_cast<const uint16_t *>(dt);
    p.b = static_cast<const uint16_t *>(b);
    p.c = static_cast<const uint16_t *>(c);
    p.out = static_cast<uint16_t *>(out);
    p.xs = x_stride;
    p.dts = dt_stride;
    p.bs = b_stride;
    p.cs = c_stride;
    p.os = out_stride;
    p.A_log = A_log;
    p.D = D;
    p.dt_bias = dt_bias;
    p.init = p.fin = state;
    p.init_dtype = p.fin_dtype = state_dtype;
    p.T = 1;
    p.H = static_cast<int>(H);
    p.P = static_cast<int>(P);
    p.G = static_cast<int>(G);
    p.nseq = static_cast<int>(S);
    p.total = static_cast<int>(S);
    return blk::launch_ssm_steps(p, static_cast<cudaStream_t>(stream));
}

KDA_API kda_status kda_gated_norm(const void *x, int64_t x_stride, const void *gate, int64_t gate_stride, const float *weight,
                                  int64_t weight_rows, void *out, int64_t out_stride, float eps, kda_act act, int gate_first,
                                  int64_t M, int64_t R, int64_t D, void *stream)
{
    t_last_error.clear();
    if (D < 8 || D % 8 || D > norm::MAX_D) return fail(KDA_ERR_SHAPE, "D must be a multiple of 8 in 8..%d (got %lld)", norm::MAX_D, (long long)D);
    if (M < 0 || M > (int64_t(1) << 31) || R < 1 || R > (1 << 20) || M * R > (int64_t(1) << 40)) return fail(KDA_ERR_SHAPE, "bad sizes M=%lld R=%lld", (long long)M, (long long)R);
    if (weight && weight_rows != 1 && weight_rows != R) return fail(KDA_ERR_SHAPE, "weight_rows must be 1 or R (got %lld)", (long long)weight_rows);
    if (!blk::act_ok(act)) return fail(KDA_ERR_RANGE, "unknown act %d", static_cast<int>(act));
    if (!std::isfinite(eps) || eps < 0.f) return fail(KDA_ERR_RANGE, "eps must be finite and not negative");
    if (M == 0) return KDA_OK;
    if (!x || !gate || !out) return fail(KDA_ERR_NULL, "x, gate and out are required");
    if (!blk::stride_ok(x_stride, R * D, 8) || !blk::stride_ok(gate_stride, R * D, 8) || !blk::stride_ok(out_stride, R * D, 8))
        return fail(KDA_ERR_ALIGN, "token strides must be multiples of 8 elements and at least R * D");
    if (!aligned(x, 16) || !aligned(gate, 16) || !aligned(out, 16) || !aligned(weight, 16))
        return fail(KDA_ERR_ALIGN, "x, gate, out and weight must be 16-byte aligned");
    const blk::Rows orow{out, 2 * out_stride, 2 * R * D, M}, xr{x, 2 * x_stride, 2 * R * D, M}, zr{gate, 2 * gate_stride, 2 * R * D, M};
    if ((!blk::same(orow, xr) && blk::share(orow, xr)) || (!blk::same(orow, zr) && blk::share(orow, zr)))
        return fail(KDA_ERR_STATE_MISMATCH, "out must be x, gate, or share no memory with them");
    if (const kda_status st = blk::check_apart({"out", orow}, {{"weight", blk::block(weight, 4 * weight_rows * D)}}); st != KDA_OK) return st;
    blk::Device d;
    if (const kda_status st = blk::device(&d); st != KDA_OK) return st;
    norm::GatedParams p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.z = static_cast<const uint16_t *>(gate);
    p.out = static_cast<uint16_t *>(out);
    p.w = weight;
    p.xs = x_stride;
    p.zs = gate_stride;
    p.os = out_stride;
    p.rows = M * R;
    p.R = static_cast<int>(R);
    p.D = static_cast<int>(D);
    p.w_rows = weight_rows == 1 ? 1 : static_cast<int>(R);
    p.eps = eps;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const blk::RowShape sh = blk::row_shape(D, p.rows, d.sms);
    if (sh.cta) return sh.vpt == 2 ? blk::launch_gated<2, true>(p, act, gate_first != 0, sh, d, s) : blk::launch_gated<4, true>(p, act, gate_first != 0, sh, d, s);
    return sh.vpt == 1   ? blk::launch_gated<1, false>(p, act, gate_first != 0, sh, d, s)
           : sh.vpt == 2 ? blk::launch_gated<2, false>(p, act, gate_first != 0, sh, d, s)
                         : blk::launch_gated<4, false>(p, act, gate_first != 0, sh, d, s);
}

KDA_API kda_status kda_residual_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                                     void *residual_out, int64_t residual_out_stride, kda_dtype residual_dtype,
                                     const void *gate, int64_t gate_stride, kda_act act, const float *post_weight,
                                     const float *channel_scale, float alpha, const float *weight, void *out,
                                     int64_t out_stride, float eps, int64_t M, int64_t D, void *stream)
{
    t_last_error.clear();
    if (D < 8 || D % 8 || D > norm::MAX_D) return fail(KDA_ERR_SHAPE, "D must be a multiple of 8 in 8..%d (got %lld)", norm::MAX_D, (long long)D);
    if (M < 0 || M > (int64_t(1) << 31)) return fail(KDA_ERR_SHAPE, "bad size M=%lld", (long long)M);
    if (residual_dtype != KDA_DTYPE_BF16 && residual_dtype != KDA_DTYPE_FP32) return fail(KDA_ERR_DTYPE, "residual dtype must be BF16 or FP32");
    if (!blk::act_ok(act)) return fail(KDA_ERR_RANGE, "unknown act %d", static_cast<int>(act));
    if (!std::isfinite(eps) || eps < 0.f) return fail(KDA_ERR_RANGE, "eps must be finite and not negative");
    if (!std::isfinite(alpha)) return fail(KDA_ERR_RANGE, "alpha must be finite");
    if (M == 0) return KDA_OK;
    if (!x || !residual || (!residual_out && !out)) return fail(KDA_ERR_NULL, "x, residual and one of residual_out and out are required");
    const int64_t rb = residual_dtype == KDA_DTYPE_FP32 ? 4 : 2, rm = 16 / rb;
    if (!blk::stride_ok(x_stride, D, 8) || !blk::stride_ok(residual_stride, D, rm) || (residual_out && !blk::stride_ok(residual_out_stride, D, rm)) ||
        (gate && !blk::stride_ok(gate_stride, D, 8)) || (out && !blk::stride_ok(out_stride, D, 8)))
        return fail(KDA_ERR_ALIGN, "row strides must be multiples of 16 bytes and at least D");
    const void *need16[] = {x, residual, residual_out, gate, out, post_weight, channel_scale, weight};
    for (const void *ptr : need16)
        if (!aligned(ptr, 16)) return fail(KDA_ERR_ALIGN, "every buffer must be 16-byte aligned");
    const blk::Rows xr{x, 2 * x_stride, 2 * D, M}, rr{residual, rb * residual_stride, rb * D, M}, zr{gate, 2 * gate_stride, 2 * D, M};
    const blk::Rows orow{out, 2 * out_stride, 2 * D, M}, ror{residual_out, rb * residual_out_stride, rb * D, M};
    auto clash = [](const blk::Rows &w, const blk::Rows &r) { return !blk::same(w, r) && blk::share(w, r); };
    if (clash(orow, xr) || clash(orow, zr) || blk::share(orow, rr) || blk::share(orow, ror) || clash(ror, rr) ||
        blk::share(ror, xr) || blk::share(ror, zr))
        return fail(KDA_ERR_STATE_MISMATCH, "out may be x or gate and residual_out may be residual; no other buffers share memory");
    {
        const blk::Named pw{"post_weight", blk::block(post_weight, 4 * D)}, ch{"channel_scale", blk::block(channel_scale, 4 * D)}, w{"weight", blk::block(weight, 4 * D)};
        if (const kda_status st = blk::check_apart({"out", orow}, {pw, ch, w}); st != KDA_OK) return st;
        if (const kda_status st = blk::check_apart({"residual_out", ror}, {pw, ch, w}); st != KDA_OK) return st;
    }
    blk::Device d;
    if (const kda_status st = blk::device(&d); st != KDA_OK) return st;
    norm::ResidualParams p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.z = static_cast<const uint16_t *>(gate);
    p.r = residual;
    p.ro = residual_out;
    p.out = static_cast<uint16_t *>(out);
    p.post = post_weight;
    p.chan = channel_scale;
    p.w = weight;
    p.xs = x_stride;
    p.zs = gate_stride;
    p.rs = residual_stride;
    p.ros = residual_out_stride;
    p.os = out_stride;
    p.rows = M;
    p.D = static_cast<int>(D);
    p.act = act;
    p.alpha = alpha;
    p.eps = eps;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = residual_dtype == KDA_DTYPE_FP32;
    const blk::RowShape sh = blk::row_shape(D, p.rows, d.sms);
    if (sh.cta) return sh.vpt == 2 ? blk::launch_residual<2, true>(p, f32, sh, d, s) : blk::launch_residual<4, true>(p, f32, sh, d, s);
    return sh.vpt == 1   ? blk::launch_residual<1, false>(p, f32, sh, d, s)
           : sh.vpt == 2 ? blk::launch_residual<2, false>(p, f32, sh, d, s)
                         : blk::launch_residual<4, false>(p, f32, sh, d, s);
}

}  // extern "C"
