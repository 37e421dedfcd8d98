// kda_mixer_api.cuh -- host side of the mixers beside KDA (include/kda.h): gated delta rule, query and key norm with
// rotation, paged cache and the attention of single tokens over it. Included by kda_fwd.cu after kda_block_api.cuh,
// whose checks it uses.
#pragma once
#include "kda_attn.cuh"
#include "kda_gdn_step.cuh"
#include "kda_gdn_tc.cuh"
#include "kda_rope.cuh"

namespace kda {
namespace mix {

using blk::block;
using blk::check_apart;
using blk::Named;
using blk::Rows;
using blk::stride_ok;

// The token-strided buffers of a delta-rule call.
struct GdnBuffers {
    Named q, k, v, a, beta, A_log, dt_bias, out, cu;
    GdnBuffers(const gdn::GdnParams &p, int64_t N)
        : q{"q", {p.q, 2 * p.qs, 2 * DH * int64_t(p.HK), p.total}}, k{"k", {p.k, 2 * p.ks, 2 * DH * int64_t(p.HK), p.total}},
          v{"v", {p.v, 2 * p.vs, 2 * DH * int64_t(p.H), p.total}}, a{"a", {p.a, 2 * p.as, 2 * int64_t(p.H), p.total}},
          beta{"beta", {p.beta, 2 * p.bs, 2 * int64_t(p.H), p.total}}, A_log{"A_log", block(p.A_log, 4 * int64_t(p.H))},
          dt_bias{"dt_bias", block(p.dt_bias, 4 * int64_t(p.H))}, out{"out", {p.out, 2 * p.os, 2 * DH * int64_t(p.H), p.total}},
          cu(blk::bounds_of(p.cu, N))
    {
    }
    kda_status check_out(const Named &state) const { return check_apart(out, {q, k, v, a, beta, A_log, dt_bias, cu, state}); }
    kda_status check_state(const Named &state) const { return check_apart(state, {q, k, v, a, beta, A_log, dt_bias, cu, out}); }
};

static kda_status check_gdn(const gdn::GdnParams &p, int64_t H, int64_t HK, int64_t K, int64_t V, uint32_t flags, bool tokens)
{
    if (K != DH || V != DH) return fail(KDA_ERR_SHAPE, "K and V must be 128 (got %lld, %lld)", (long long)K, (long long)V);
    if (H < 1 || H > (1 << 20) || HK < 1 || H % HK) return fail(KDA_ERR_SHAPE, "HK must divide H (H=%lld HK=%lld)", (long long)H, (long long)HK);
    if (flags & ~KDA_FLAG_QK_L2NORM) return fail(KDA_ERR_RANGE, "unknown flags 0x%x", flags);
    if (!std::isfinite(p.scale)) return fail(KDA_ERR_RANGE, "scale must be finite");
    if (!p.A_log || (tokens && (!p.q || !p.k || !p.v || !p.a || !p.beta || !p.out)))
        return fail(KDA_ERR_NULL, "q, k, v, a, beta, A_log and out are required");
    if (!aligned(p.A_log, 4) || !aligned(p.dt_bias, 4)) return fail(KDA_ERR_ALIGN, "A_log and dt_bias must be 4-byte aligned");
    if (!tokens) return KDA_OK;
    if (!stride_ok(p.qs, HK * DH, 8) || !stride_ok(p.ks, HK * DH, 8) || !stride_ok(p.vs, H * DH, 8) || !stride_ok(p.os, H * DH, 8) ||
        !stride_ok(p.as, H, 1) || !stride_ok(p.bs, H, 1))
        return fail(KDA_ERR_ALIGN, "token strides must cover a token's elements and, but for a's and beta's, be multiples of 8 elements");
    if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.out, 16) || !aligned(p.a, 2) || !aligned(p.beta, 2))
        return fail(KDA_ERR_ALIGN, "q, k, v and out must be 16-byte, a and beta 2-byte aligned");
    return KDA_OK;
}

static gdn::GdnParams gdn_params(const void *q, int64_t qs, const void *k, int64_t ks, const void *v, int64_t vs, const void *a, int64_t as,
                                 const void *beta, int64_t bs, float scale, void *out, int64_t os, const float *A_log, const float *dt_bias,
                                 uint32_t flags)
{
    gdn::GdnParams p = {};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.a = static_cast<const uint16_t *>(a);
    p.beta = static_cast<const uint16_t *>(beta);
    p.out = static_cast<uint16_t *>(out);
    p.qs = qs;
    p.ks = ks;
    p.vs = vs;
    p.as = as;
    p.bs = bs;
    p.os = os;
    p.A_log = A_log;
    p.dt_bias = dt_bias;
    p.scale = scale;
    p.l2 = (flags & KDA_FLAG_QK_L2NORM) != 0;
    return p;
}

static kda_status launch_gdn_steps(const gdn::GdnParams &p, cudaStream_t s)
{
    const int64_t warps = static_cast<int64_t>(p.nseq) * p.H * (DH / gdn::ROWS);
    const int64_t grid = (warps + gdn::STEP_THREADS / 32 - 1) / (gdn::STEP_THREADS / 32);
    gdn::kda_gdn_step_kernel<<<static_cast<unsigned>(grid), gdn::STEP_THREADS, 0, s>>>(p, warps);
    return blk::launched("gated delta rule step");
}

static kda_status launch_gdn_tc(const gdn::GdnParams &p, cudaStream_t s)
{
    CUtensorMap mq, mk, mv, mo;
    if (!blk::rows_map(&mq, p.q, p.total, p.HK, DH, p.qs, gdntc::C) || !blk::rows_map(&mk, p.k, p.total, p.HK, DH, p.ks, gdntc::C) ||
        !blk::rows_map(&mv, p.v, p.total, p.H, DH, p.vs, gdntc::C) || !blk::rows_map(&mo, p.out, p.total, p.H, DH, p.os, gdntc::C))
        return fail(KDA_ERR_LAUNCH, "cuTensorMapEncodeTiled failed (driver entry point unavailable or bad geometry)");
    static thread_local int configured_dev = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_dev != dev) {
        const cudaError_t e = cudaFuncSetAttribute(gdntc::kda_gdn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, gdntc::Layout::ALLOC);
        if (e != cudaSuccess) return fail(KDA_ERR_LAUNCH, "gated delta rule set-up failed: %s", cudaGetErrorString(e));
        configured_dev = dev;
    }
    gdntc::kda_gdn_tc_kernel<<<static_cast<unsigned>(p.nseq * static_cast<int64_t>(p.H)), gdntc::NTHREADS, gdntc::Layout::ALLOC, s>>>(mq, mk, mv, mo, p);
    return blk::launched("gated delta rule");
}

// What qk_rope and kv_append share: the turn and the norm of heads of D channels.
static kda_status check_turn(const int64_t *positions, const float *inv_freq, int64_t R, int norm, float eps, int64_t D)
{
    if (D != 64 && D != 128 && D != 256) return fail(KDA_ERR_SHAPE, "D must be 64, 128 or 256 (got %lld)", (long long)D);
    if (R < 0 || R > D || R % 16) return fail(KDA_ERR_SHAPE, "R must be a multiple of 16 in 0..D (got %lld)", (long long)R);
    if (R > 0 && !inv_freq) return fail(KDA_ERR_NULL, "inv_freq is required where channels are turned");
    if (norm && (!std::isfinite(eps) || eps < 0.f)) return fail(KDA_ERR_RANGE, "eps must be finite and not negative");
    if (!aligned(positions, 8) || !aligned(inv_freq, 4)) return fail(KDA_ERR_ALIGN, "positions must be 8-byte and inv_freq 4-byte aligned");
    return KDA_OK;
}

static rope::Turn turn_of(const int64_t *positions, const float *inv_freq, int64_t R, int interleaved)
{
    return {positions, inv_freq, static_cast<int>(R), interleaved != 0};
}

static kda_status check_pages(const void *k_cache, const void *v_cache, int64_t page_stride, int64_t pages, int64_t page_size,
                              const int32_t *table, int64_t width, int64_t HK, int64_t D)
{
    if (page_size < 8 || page_size > 4096 || (page_size & (page_size - 1)))
        return fail(KDA_ERR_SHAPE, "page_size must be a power of two in 8..4096 (got %lld)", (long long)page_size);
    if (pages < 1 || pages > (int64_t(1) << 30) || width < 1 || width > (int64_t(1) << 28))
        return fail(KDA_ERR_SHAPE, "bad sizes pages=%lld table width=%lld", (long long)pages, (long long)width);
    if (!k_cache || !v_cache || !table) return fail(KDA_ERR_NULL, "k_cache, v_cache and page_table are required");
    if (!stride_ok(page_stride, HK * page_size * D, 8)) return fail(KDA_ERR_ALIGN, "page_stride must be a multiple of 8 elements and at least HK * page_size * D");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(table, 4)) return fail(KDA_ERR_ALIGN, "caches must be 16-byte, page_table 4-byte aligned");
    return KDA_OK;
}

// go(width, interleaved) with both as constants
template <class Go>
static void by_width(int64_t D, bool interleaved, const Go &go)
{
    auto pairs = [&](auto d) { interleaved ? go(d, std::true_type()) : go(d, std::false_type()); };
    D == 64 ? pairs(std::integral_constant<int, 64>()) : D == 128 ? pairs(std::integral_constant<int, 128>()) : pairs(std::integral_constant<int, 256>());
}

static rope::Pages pages_of(int64_t page_stride, int64_t pages, int64_t page_size, const int32_t *table, int64_t width)
{
    int shift = 0;
    while ((int64_t(1) << shift) < page_size) ++shift;
    return {page_stride, table, static_cast<int>(width), static_cast<int>(pages), shift};
}

// Warps with a run of the cache, and the workspace with which runs may be cut inside a unit.
static int64_t attn_workers(int sms) { return static_cast<int64_t>(sms) * attn::CTAS * attn::WARPS; }
static size_t attn_bytes(int64_t D, int sms) { return static_cast<size_t>(attn_workers(sms)) * 2 * 16 * (D + 2) * sizeof(float); }

template <int D>
static kda_status launch_attn(const attn::AttnParams &p, cudaStream_t s)
{
    static thread_local int configured_dev = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_dev != dev) {
        const cudaError_t e = cudaFuncSetAttribute(attn::kda_attn_step_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, attn::smem_of(D));
        if (e != cudaSuccess) return fail(KDA_ERR_LAUNCH, "attention set-up failed: %s", cudaGetErrorString(e));
        configured_dev = dev;
    }
    attn::kda_attn_step_kernel<D><<<(p.workers + attn::WARPS - 1) / attn::WARPS, attn::THREADS, attn::smem_of(D), s>>>(p);
    if (const kda_status st = blk::launched("attention step"); st != KDA_OK || !p.ws) return st;
    // few units are looked at one by one, with a block for each of their rows; many at the borders between the runs
    const int64_t units = static_cast<int64_t>(p.S) * p.HK * p.tiles;
    const bool by_unit = units <= p.workers;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(by_unit ? units : p.workers - 1), static_cast<unsigned>(units <= 64 ? std::min(p.rows, 16) : 1));
    cfg.blockDim = dim3(attn::JOIN_THREADS);
    cfg.dynamicSmemBytes = cfg.blockDim.x / 32 * (D + 2) * sizeof(float);
    cfg.stream = s;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its blocks look for their unit while the last runs end
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn::kda_attn_join_kernel<D>, p, static_cast<int>(by_unit));
    if (e != cudaSuccess) return fail(KDA_ERR_LAUNCH, "attention join launch failed: %s", cudaGetErrorString(e));
    return KDA_OK;
}

// Tokens per CTA: one while CTAs are fewer than the machine takes at once, up to `limit`.
static int tokens_per_cta(int64_t M, int sms, int limit)
{
    int n = 1;
    while (n < limit && M > static_cast<int64_t>(sms) * 8 * n) n <<= 1;
    return n;
}

}  // namespace mix
}  // namespace kda

extern "C" {

KDA_API kda_status kda_gdn(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                           const void *a, int64_t a_stride, const void *beta, int64_t beta_stride, float scale, void *out,
                           int64_t out_stride, const float *A_log, const float *dt_bias, const void *initial_state,
                           kda_dtype initial_dtype, void *final_state, kda_dtype final_dtype, const int64_t *cu_seqlens,
                           int64_t N, int64_t B, int64_t T, int64_t H, int64_t HK, int64_t K, int64_t V, uint32_t flags, void *stream)
{
    t_last_error.clear();
    int64_t nseq = 0, total = 0;
    if (const kda_status st = blk::check_varlen(cu_seqlens, N, B, T, &nseq, &total); st != KDA_OK) return st;
    gdn::GdnParams p = mix::gdn_params(q, q_stride, k, k_stride, v, v_stride, a, a_stride, beta, beta_stride, scale, out, out_stride,
                                       A_log, dt_bias, flags);
    if (const kda_status st = mix::check_gdn(p, H, HK, K, V, flags, total > 0); st != KDA_OK) return st;
    if (nseq * H > (int64_t(1) << 26)) return fail(KDA_ERR_SHAPE, "too many (sequence, head) pairs");
    auto dt_ok = [](const void *ptr, kda_dtype d) {
        return ptr ? (d == KDA_DTYPE_BF16 || d == KDA_DTYPE_FP32) : d == KDA_DTYPE_NONE;
    };
    if (!dt_ok(initial_state, initial_dtype) || !dt_ok(final_state, final_dtype))
        return fail(KDA_ERR_DTYPE, "state dtype codes must be BF16/FP32 for a given buffer and NONE for an absent one");
    if (!aligned(initial_state, 16) || !aligned(final_state, 16)) return fail(KDA_ERR_ALIGN, "state buffers must be 16-byte aligned");
    auto state_block = [&](const void *ptr, kda_dtype d) { return blk::block(ptr, nseq * H * DH * DH * (d == KDA_DTYPE_FP32 ? 4 : 2)); };
    if (initial_state && final_state) {
        if (initial_dtype != final_dtype) return fail(KDA_ERR_STATE_MISMATCH, "final_state must match initial_state's dtype");
        if (blk::partial_overlap(initial_state, final_state, state_block(initial_state, initial_dtype).width))
            return fail(KDA_ERR_STATE_MISMATCH, "initial_state and final_state overlap partially");
    }
    p.init = initial_state;
    p.fin = final_state;
    p.cu = cu_seqlens;
    p.init_dtype = initial_dtype;
    p.fin_dtype = final_dtype;
    p.T = static_cast<int>(T);
    p.H = static_cast<int>(H);
    p.HK = static_cast<int>(HK);
    p.nseq = static_cast<int>(nseq);
    p.total = static_cast<int>(total);
    const mix::GdnBuffers bufs(p, N);
    if (const kda_status st = bufs.check_out({"initial_state", state_block(initial_state, initial_dtype)}); st != KDA_OK) return st;
    if (const kda_status st = bufs.check_state({"final_state", state_block(final_state, final_dtype)}); st != KDA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (total <= (cu_seqlens ? 1 : nseq) * gdn::STEP_TOKENS) return mix::launch_gdn_steps(p, s);
    // A packed call's short sequences are walked by the chunk kernel's CTAs, one to an SM, or, where the lengths are short in
    // the mean, by a launch of their own ahead of it. us for 128 sequences of 16 heads, by the one and the other: single tokens
    // 106, 52; 8 tokens each 227, 130; these and one of 1024 tokens 227, 175; 9 tokens each, where none is short, 134, 143. One of
    // 4096 tokens and 128 single ones: 157 by the CTAs, no more than the 4096 alone.
    p.split = cu_seqlens && total <= nseq * 2 * gdn::STEP_TOKENS;
    if (p.split)
        if (const kda_status st = mix::launch_gdn_steps(p, s); st != KDA_OK) return st;
    return mix::launch_gdn_tc(p, s);
}

KDA_API kda_status kda_gdn_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                const void *a, int64_t a_stride, const void *beta, int64_t beta_stride, float scale, void *out,
                                int64_t out_stride, const float *A_log, const float *dt_bias, void *state, kda_dtype state_dtype,
                                int64_t S, int64_t H, int64_t HK, int64_t K, int64_t V, uint32_t flags, void *stream)
{
    t_last_error.clear();
    if (S < 1 || H < 1 || S > (int64_t(1) << 26) || H > (int64_t(1) << 26) || S * H > (int64_t(1) << 26))
        return fail(KDA_ERR_SHAPE, "bad sizes S=%lld H=%lld", (long long)S, (long long)H);
    gdn::GdnParams p = mix::gdn_params(q, q_stride, k, k_stride, v, v_stride, a, a_stride, beta, beta_stride, scale, out, out_stride,
                                       A_log, dt_bias, flags);
    if (const kda_status st = mix::check_gdn(p, H, HK, K, V, flags, true); st != KDA_OK) return st;
    if (!state) return fail(KDA_ERR_NULL, "state is required");
    if (state_dtype != KDA_DTYPE_BF16 && state_dtype != KDA_DTYPE_FP32) return fail(KDA_ERR_DTYPE, "state dtype must be BF16 or FP32");
    if (!aligned(state, 16)) return fail(KDA_ERR_ALIGN, "state must be 16-byte aligned");
    p.init = p.fin = state;
    p.init_dtype = p.fin_dtype = state_dtype;
    p.T = 1;
    p.H = static_cast<int>(H);
    p.HK = static_cast<int>(HK);
    p.nseq = p.total = static_cast<int>(S);
    const mix::GdnBuffers bufs(p, 0);
    const blk::Named st_buf{"state", blk::block(state, S * H * DH * DH * (state_dtype == KDA_DTYPE_FP32 ? 4 : 2))};
    if (const kda_status st = bufs.check_out(st_buf); st != KDA_OK) return st;
    if (const kda_status st = bufs.check_state(st_buf); st != KDA_OK) return st;
    return mix::launch_gdn_steps(p, static_cast<cudaStream_t>(stream));
}

KDA_API kda_status kda_qk_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, void *q_out, int64_t q_out_stride,
                               void *k_out, int64_t k_out_stride, const float *q_weight, const float *k_weight, int norm, float eps,
                               const int64_t *positions, const float *inv_freq, int64_t R, int interleaved, int64_t M, int64_t H,
                               int64_t HK, int64_t D, void *stream)
{
    t_last_error.clear();
    if (M < 0 || M > (int64_t(1) << 31) || H < 1 || H > (1 << 16) || HK < 0 || HK > (1 << 16))
        return fail(KDA_ERR_SHAPE, "bad sizes M=%lld H=%lld HK=%lld", (long long)M, (long long)H, (long long)HK);
    if (const kda_status st = mix::check_turn(positions, inv_freq, R, norm, eps, D); st != KDA_OK) return st;
    if (M == 0) return KDA_OK;
    if (!q || !q_out || !positions || (HK > 0 && (!k || !k_out))) return fail(KDA_ERR_NULL, "q, q_out, positions and, for HK > 0, k and k_out are required");
    if (!blk::stride_ok(q_stride, H * D, 8) || !blk::stride_ok(q_out_stride, H * D, 8) ||
        (HK > 0 && (!blk::stride_ok(k_stride, HK * D, 8) || !blk::stride_ok(k_out_stride, HK * D, 8))))
        return fail(KDA_ERR_ALIGN, "token strides must be multiples of 8 elements and cover a token's elements");
    const void *need16[] = {q, q_out, k, k_out, q_weight, k_weight};
    for (const void *ptr : need16)
        if (!aligned(ptr, 16)) return fail(KDA_ERR_ALIGN, "q, k, their outputs and weights must be 16-byte aligned");
    if (HK == 0) k = k_out = nullptr;
    const blk::Rows qr{q, 2 * q_stride, 2 * H * D, M}, kr{k, 2 * k_stride, 2 * HK * D, M}, qo{q_out, 2 * q_out_stride, 2 * H * D, M},
        ko{k_out, 2 * k_out_stride, 2 * HK * D, M};
    if ((!blk::same(qo, qr) && blk::share(qo, qr)) || blk::share(qo, kr) || blk::share(qo, ko) || blk::share(ko, qr) ||
        (!blk::same(ko, kr) && blk::share(ko, kr)))
        return fail(KDA_ERR_STATE_MISMATCH, "q_out may be q and k_out may be k; no other buffers share memory");
    for (const blk::Named &w : {blk::Named{"q_out", qo}, blk::Named{"k_out", ko}})
        if (const kda_status st = blk::check_apart(w, {{"q_weight", blk::block(q_weight, 4 * D)}, {"k_weight", blk::block(k_weight, 4 * D)},
                                                       {"positions", blk::block(positions, 8 * M)}, {"inv_freq", blk::block(R ? inv_freq : nullptr, 2 * R)}});
            st != KDA_OK)
            return st;
    blk::Device d;
    if (const kda_status st = blk::device(&d); st != KDA_OK) return st;
    rope::QkParams p = {};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.qo = static_cast<uint16_t *>(q_out);
    p.ko = static_cast<uint16_t *>(k_out);
    p.qs = q_stride;
    p.ks = k_stride;
    p.qos = q_out_stride;
    p.kos = k_out_stride;
    p.qw = q_weight;
    p.kw = k_weight;
    p.turn = mix::turn_of(positions, inv_freq, R, interleaved);
    p.hn = {norm != 0, eps};
    p.M = M;
    p.H = static_cast<int>(H);
    p.HK = static_cast<int>(HK);
    p.tokens = mix::tokens_per_cta(M, d.sms, rope::MAX_TOKENS);
    const unsigned grid = static_cast<unsigned>((M + p.tokens - 1) / p.tokens);
    const size_t table = static_cast<size_t>(p.tokens) * (R / 2) * sizeof(float2);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    mix::by_width(D, interleaved != 0, [&](auto d, auto inter) {
        rope::kda_qk_rope_kernel<decltype(d)::value, decltype(inter)::value><<<grid, rope::THREADS, table, s>>>(p);
    });
    return blk::launched("query and key rotation");
}

KDA_API kda_status kda_kv_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *k_cache, void *v_cache,
                                 int64_t page_stride, int64_t pages, int64_t page_size, const int32_t *page_table, int64_t table_width,
                                 const int64_t *positions, const float *inv_freq, int64_t R, int interleaved, const float *k_weight,
                                 int norm, float eps, const int64_t *cu_seqlens, int64_t N, int64_t B, int64_t T, int64_t HK, int64_t D,
                                 void *stream)
{
    t_last_error.clear();
    int64_t nseq = 0, M = 0;
    if (const kda_status st = blk::check_varlen(cu_seqlens, N, B, T, &nseq, &M); st != KDA_OK) return st;
    if (HK < 1 || HK > (1 << 16)) return fail(KDA_ERR_SHAPE, "bad size HK=%lld", (long long)HK);
    if (const kda_status st = mix::check_turn(positions, inv_freq, R, norm, eps, D); st != KDA_OK) return st;
    if (const kda_status st = mix::check_pages(k_cache, v_cache, page_stride, pages, page_size, page_table, table_width, HK, D); st != KDA_OK) return st;
    if (M == 0) return KDA_OK;
    if (!k || !v || !positions) return fail(KDA_ERR_NULL, "k, v and positions are required");
    if (!blk::stride_ok(k_stride, HK * D, 8) || !blk::stride_ok(v_stride, HK * D, 8))
        return fail(KDA_ERR_ALIGN, "token strides must be multiples of 8 elements and cover a token's elements");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_weight, 16)) return fail(KDA_ERR_ALIGN, "k, v and k_weight must be 16-byte aligned");
    const blk::Rows kc{k_cache, 2 * page_stride, 2 * HK * page_size * D, pages}, vc{v_cache, 2 * page_stride, 2 * HK * page_size * D, pages};
    if (blk::share(kc, vc)) return fail(KDA_ERR_STATE_MISMATCH, "k_cache and v_cache must not share memory");
    for (const blk::Named &c : {blk::Named{"k_cache", kc}, blk::Named{"v_cache", vc}})
        if (const kda_status st = blk::check_apart(c, {{"k", {k, 2 * k_stride, 2 * HK * D, M}}, {"v", {v, 2 * v_stride, 2 * HK * D, M}},
                                                       {"page_table", blk::block(page_table, 4 * nseq * table_width)},
                                                       {"positions", blk::block(positions, 8 * M)}, {"k_weight", blk::block(k_weight, 4 * D)},
                                                       {"inv_freq", blk::block(R ? inv_freq : nullptr, 2 * R)}, blk::bounds_of(cu_seqlens, N)});
            st != KDA_OK)
            return st;
    blk::Device d;
    if (const kda_status st = blk::device(&d); st != KDA_OK) return st;
    rope::AppendParams p = {};
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.kc = static_cast<uint16_t *>(k_cache);
    p.vc = static_cast<uint16_t *>(v_cache);
    p.ks = k_stride;
    p.vs = v_stride;
    p.kw = k_weight;
    p.turn = mix::turn_of(positions, inv_freq, R, interleaved);
    p.hn = {norm != 0, eps};
    p.pages = mix::pages_of(page_stride, pages, page_size, page_table, table_width);
    p.cu = cu_seqlens;
    p.M = M;
    p.T = static_cast<int>(T);
    p.nseq = static_cast<int>(nseq);
    p.HK = static_cast<int>(HK);
    p.tokens = mix::tokens_per_cta(M, d.sms, rope::MAX_TOKENS / 2);
    const unsigned grid = static_cast<unsigned>((M + p.tokens - 1) / p.tokens);
    const size_t table = static_cast<size_t>(p.tokens) * (R / 2) * sizeof(float2);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    mix::by_width(D, interleaved != 0, [&](auto d, auto inter) {
        rope::kda_kv_append_kernel<decltype(d)::value, decltype(inter)::value><<<grid, rope::THREADS, table, s>>>(p);
    });
    return blk::launched("cache append");
}

KDA_API kda_status kda_attn_step_workspace_bytes(int64_t S, int64_t H, int64_t HK, int64_t D, size_t *bytes)
{
    t_last_error.clear();
    if (!bytes) return fail(KDA_ERR_NULL, "kda_attn_step_workspace_bytes: bytes is required");
    if (S < 0 || HK < 1 || H < 1 || H % HK || (D != 64 && D != 128))
        return fail(KDA_ERR_SHAPE, "bad sizes S=%lld H=%lld HK=%lld D=%lld", (long long)S, (long long)H, (long long)HK, (long long)D);
    blk::Device d;
    if (const kda_status st = blk::device(&d); st != KDA_OK) return st;
    *bytes = S > 0 ? mix::attn_bytes(D, d.sms) : 0;
    return KDA_OK;
}

KDA_API kda_status kda_attn_step(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache, int64_t page_stride,
                                 int64_t pages, int64_t page_size, const int32_t *page_table, int64_t table_width,
                                 const int64_t *positions, float scale, void *out, int64_t out_stride, float *lse, int64_t S, int64_t H,
                                 int64_t HK, int64_t D, void *workspace, size_t workspace_bytes, void *stream)
{
    t_last_error.clear();
    if (S < 1 || S > (1 << 16) || HK < 1 || H < 1 || H > (1 << 16) || H % HK)
        return fail(KDA_ERR_SHAPE, "HK must divide H (S=%lld H=%lld HK=%lld)", (long long)S, (long long)H, (long long)HK);
    if (D != 64 && D != 128) return fail(KDA_ERR_SHAPE, "D must be 64 or 128 (got %lld)", (long long)D);
    if (const kda_status st = mix::check_pages(k_cache, v_cache, page_stride, pages, page_size, page_table, table_width, HK, D); st != KDA_OK) return st;
    if (!std::isfinite(scale)) return fail(KDA_ERR_RANGE, "scale must be finite");
    if (!q || !positions || !out) return fail(KDA_ERR_NULL, "q, positions and out are required");
    if (!blk::stride_ok(q_stride, H * D, 8) || !blk::stride_ok(out_stride, H * D, 8))
        return fail(KDA_ERR_ALIGN, "row strides must be multiples of 8 elements and at least H * D");
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(positions, 8) || !aligned(lse, 4) || !aligned(workspace, 16))
        return fail(KDA_ERR_ALIGN, "q, out and workspace must be 16-byte, positions 8-byte, lse 4-byte aligned");
    const blk::Named qr{"q", {q, 2 * q_stride, 2 * H * D, S}}, orow{"out", {out, 2 * out_stride, 2 * H * D, S}}, lr{"lse", blk::block(lse, 4 * S * H)};
    const blk::Named kc{"k_cache", {k_cache, 2 * page_stride, 2 * HK * page_size * D, pages}}, vc{"v_cache", {v_cache, 2 * page_stride, 2 * HK * page_size * D, pages}};
    const blk::Named tab{"page_table", blk::block(page_table, 4 * S * table_width)}, pos{"positions", blk::block(positions, 8 * S)};
    if (const kda_status st = blk::check_apart(orow, {qr, kc, vc, tab, pos, lr}); st != KDA_OK) return st;
    if (const kda_status st = blk::check_apart(lr, {qr, kc, vc, tab, pos}); st != KDA_OK) return st;
    attn::AttnParams p = {};
    p.q = static_cast<const uint16_t *>(q);
    p.kc = static_cast<const uint16_t *>(k_cache);
    p.vc = static_cast<const uint16_t *>(v_cache);
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.qs = q_stride;
    p.os = out_stride;
    p.positions = positions;
    p.pages = mix::pages_of(page_stride, pages, page_size, page_table, table_width);
    p.scale = scale;
    p.S = static_cast<int>(S);
    p.H = static_cast<int>(H);
    p.HK = static_cast<int>(HK);
    p.D = static_cast<int>(D);
    p.rows = static_cast<int>(H / HK);
    p.tiles = (p.rows + 15) / 16;
    blk::Device d;
    if (const kda_status st = blk::device(&d); st != KDA_OK) return st;
    p.workers = static_cast<int>(mix::attn_workers(d.sms));
    if (workspace) {
        const size_t need = mix::attn_bytes(D, d.sms);
        if (workspace_bytes < need) return fail(KDA_ERR_RANGE, "workspace of %zu bytes is smaller than the %zu this call needs", workspace_bytes, need);
        const blk::Named ws{"workspace", blk::block(workspace, static_cast<int64_t>(need))};
        if (const kda_status st = blk::check_apart(ws, {qr, orow, lr, kc, vc, tab, pos}); st != KDA_OK) return st;
        p.ws = static_cast<float *>(workspace);
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return D == 64 ? mix::launch_attn<64>(p, s) : mix::launch_attn<128>(p, s);
}

}  // extern "C"
