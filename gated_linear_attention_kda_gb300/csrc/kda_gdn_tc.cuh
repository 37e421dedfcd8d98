// kda_gdn_tc.cuh -- the gated delta rule with one decay per head over prompts, on the 5th-generation tensor core, 64 tokens
// at a time.
//
// Chunk algebra. Over a chunk of tokens j = 0..63 that starts from S0 (V x K), with G_i the running sum of the log2 decays
// up to and with token i, the misses n_i = v_i - 2^(a_i) S_{i-1} k_i, of which the state takes b_i, satisfy
//   (I + A) N = V - diag(2^G) K S0^T,   A[i, j] = 2^(G_i - G_j) b_j k_i . k_j   for j < i, else 0
// so that with T = (I + A)^-1
//   N     = T V - T diag(2^G) K S0^T
//   out_i = scale (2^(G_i) S0 q_i + sum_{j <= i} 2^(G_i - G_j) b_j (q_i . k_j) n_j)
//   S1    = 2^(G_63) S0 + sum_j 2^(G_63 - G_j) b_j n_j k_j^T
// (With the steps inside T, as diag(b), its diagonal would have to be rounded: here it is one, which is exact, and it is
// most of T where keys are not alike: outputs are off by 3.1e-3 of their head's norm this way, 3.4e-3 the other.)
// No exponent is positive, so nothing overflows, and with one decay per head every scaling is by a token: K, Q and V enter
// the products as they lie in memory, and norms of queries and keys are factors of the same kind.
//
// One CTA owns the state of one (sequence, head). It lives in tensor memory, fp32, lane = value channel, column = key
// channel, and everything on the chain from chunk to chunk keeps the value channel in its lane:
//   D1  [128 x 64]  = S K^T           S as bf16 in tensor memory (its own copy)
//   D2  [128 x 64]  = V^T T^T         V^T straight from V's tile (its transpose is a layout of the operand)
//   D2             += D1' T^T         D1' = -2^(G_j) D1 as bf16, written over D1
//   S              += N' K            N' = 2^(G_63 - G_j) b_j N^T as bf16, written over D1'; S decayed before
//   O   [128 x 64]  = S Q^T,  N^T P^T and the output is their sum, the first scaled per token; N as it lies in D2, tf32
// Beside the chain, one or two chunks ahead: [K; Q] K^T, its scaled halves A and P, and T. D1' T^T and N^T P^T take 16 tokens j
// at a time, each for the outputs i from there on: T and P are zero before.
// Roundings: the state, D1', N' and T enter products as bf16, N and P as tf32, cut off by the instruction (the output is
// bf16; the state that is carried and returned is fp32). The inverse is fp32 within 8 x 8 blocks and tf32 between them
// (products rounded to nearest, A cut off by the instruction), an eighth and a quarter of the step of T's own rounding.
// What they make depends on the keys. Where these have a common direction, an output is a sum of P[i, j] n_j that take each
// other back (where all are one and steps near one it telescopes), and what each term is off by adds up. With N and P as
// bf16 outputs were off by 3.1e-3 of a head's norm for independent keys, and by 5.8e-3, 9.3e-3, 1.3e-2 for keys with a cosine of
// .3, .6, .9 between them (steps about .5, decays about .99); in tf32 they are by 2.8e-3, 3.0e-3, 4.3e-3, 6.0e-3, of which the
// output's own rounding is 1.66e-3, and the rest mostly T's and the state's. That costs twice P's shared memory (V has one
// buffer for it), and 3 % where one sequence's chain is all (4.42 to 4.57 ms for 131,072 tokens of 32 heads), 1 % for 8 x
// 4096 tokens; packed prompts take 1 % less, as N is no longer converted. A second bf16 part of T would bring them to 2.5e-3
// throughout (by an emulation). One of N' brings bf16 states of independent keys from 2.4e-3 to their own rounding, 1.7e-3, and
// outputs from 2.1e-3 to 1.95e-3, and was not kept: four more products on the chain, 8 x 4096 tokens 164 to 178 us, packed prompts
// 647 to 682, a long one 4,570 to 4,750 (of the last 32 tokens of a chunk alone: 1.8e-3 to 2.1e-3, 172, 686, 4,630). Where all keys
// of a chunk are one, steps are near one and nothing decays, what T's rows sum to for their rounding adds up: .09 after 64
// tokens.
//
// NaN: a product multiplies what a mask leaves out by zero, and 0 NaN is NaN, so a token that holds a NaN or infinity
// would reach earlier ones of its chunk. What holds one leaves no number in the state's rows it reaches, up to the end of
// the sequence, where such rows show; their eight neighbours' outputs and states are then made again token by token from
// the start of the sequence (walk_rows). A NaN in q stays in its token without that.
//
// What bounds it (8 x 4096 tokens of 16 heads: 163 us, 3.3 TB/s of 6.7; one sequence of 131,072 tokens of 32 heads: 4.6 ms,
// 2.2 us a chunk on 32 SMs; cycles as counted at 160 us, before N and P were tf32). Three loops of 4,500 to 4,700 cycles a
// chunk, about even by the clocks of their steps: the chain
// (S to bf16 500, D1 1,350, D1' 400, N 1,100, N' 450, S 700); the scores' one accumulator (product 1,600 from the wait on,
// read 3,050 by the warps with four blocks of columns); and, over two chunks, a tile's way from its load over the norms and
// the scores to T (inverse 3,500). The tensor pipe is busy 30 % of the time. Next to that, instruction supply: the
// roles' loops hold some 40 KB of code (chain and its issuer 9, the other issuers and decays 9, output and norms 10, A, P
// and T 13), which every chunk runs through once; the SM's own cache misses one fetch in thirteen and
// the port of the one behind it runs at 78 % of its peak. 8 KB more straight-line code on the chain made the kernel 11 % slower,
// unrolling the eight products of one issuer 5 %, a call in place of an inlined wait costs 200 cycles more than the wait; so
// loops over products stay rolled, waits are a few instructions, and masks are made only where they are read. Against 162 us
// in one run: the inverse's products rolled as well 164 to 176; scores read a block ahead of their use, which frees the
// accumulator sooner, 176; their factors outside diagonal blocks as a row's times a column's, which saves 30 of 64
// exponentials, 184.
// Roles were split until the chain had warps of its own (209 us with A, P and T by one group of warps, 180 with norms and
// output MMAs moved off the chain's issuers, 165 with two groups in turn, 160 with the steps outside T). Two CTAs per SM do
// not fit: tensor memory and 220 KB of shared memory are full.
//
// Warp roles (768 threads):
//   warp 0       TMA producer (lane 0): [K; Q] tiles three deep, V's one
//   warp 1       MMA issuer: the chain
//   warp 2       MMA issuer: [K; Q] K^T, V^T T^T
//   warp 3       MMA issuer: output; running sums of the decays, steps
//   warps 4-11   chain: bf16 state, D1', N and N', decay (value channel, half of the columns each)
//   warps 12-15  output (value channel), transposed on the way through shared memory; norms of queries and keys
//   warps 16-23  A, P and T of a chunk, two groups in turn
#pragma once
#include "kda_gdn_step.cuh"
#include "kda_ssm_tc.cuh"
#include "tcgen05.cuh"

namespace kda {
namespace gdntc {

using gdn::GdnParams;

constexpr int C = 64;           // tokens per chunk
constexpr int NTHREADS = 768;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t T_S = 0, T_SB = 128, T_D1 = 192, T_SQ = 256, T_D2 = 320, T_PV = 384, T_KQ = 448;

// scalars of a chunk: running log2 sums, steps, 2^G (then the factors of D1'), 2^(G_63 - G) (then those of N'), the
// output's factors; by key column G less log2 b / |k|; by row 1 / |k| and scale / |q|; the chunk's whole decay
constexpr int SC_G = 0, SC_B = 256, SC_D = 512, SC_N = 768, SC_O = 1024, SC_GK = 1280, SC_FK = 1536, SC_FQ = 1792, SC_GAM = 2048, SC_BYTES = 2064;

struct Layout {
    static constexpr int BOX = C * 128;             // 64 channels x 64 rows, 128-byte swizzle
    static constexpr int KQS = 3, KQT = 4 * BOX;    // a tile: per 64 channels the rows of K, then those of Q
    static constexpr int VT = 2 * BOX;              // one tile of V
    static constexpr int PS = KQS, PT = 2 * BOX;    // score tiles, fp32: per 32 columns 64 rows of 128 bytes
    static constexpr int TS = 2;                    // T tiles
    // the inverse's scratch, fp32, one per group: rows 0..31 need 32 columns, the others 64 (and four more for the banks)
    static constexpr int LD0 = 36, LD1 = 68, SCRATCH = 32 * (LD0 + LD1) * 4;
    static constexpr int KQ = 0;
    static constexpr int V = KQ + KQS * KQT;
    static constexpr int P = V + VT;                // scores [i][j]
    static constexpr int T = P + PS * PT;           // T [i][j], bf16, 128-byte rows
    static constexpr int SCR = T + TS * BOX;
    static constexpr int SC = SCR + 2 * SCRATCH;
    static constexpr int BAR = SC + 4 * SC_BYTES;
    static constexpr int KQ_FULL = 0, KQ_EMPTY = 3, V_FULL = 6, V_EMPTY = 7, SC_FULL = 10, T_FULL = 13, G_DONE = 35, KQ_FREE = 17,
                         KQ_ZERO = 18, SB_GO = 19, D1_DONE = 20, D1_GO = 21, N_DONE = 22, N_GO = 23, S_DONE = 24, O_DONE = 25,
                         SQ_DONE = 26, U_DONE = 27, OUT_RD = 28, FACT = 29, END = 32, END2 = 33, END3 = 34, T_EMPTY = 37, NBARS = 39;
    static constexpr int TMEMPTR = (BAR + NBARS * 8 + 15) / 16 * 16;
    static constexpr int FLAGS = TMEMPTR + 16;      // a wait ran out; groups of eight rows that hold no numbers at the end
    static constexpr int OUT = (FLAGS + 16 + 1023) / 1024 * 1024;  // a chunk's output, [token][channel]
    static constexpr int ALLOC = OUT + VT;          // all of it: the window starts on 1024 bytes, as nothing is static
    static_assert(ALLOC <= 227 * 1024, "shared memory budget");
    static_assert(SC % 16 == 0 && SC_BYTES % 16 == 0 && BAR % 8 == 0 && P % 1024 == 0 && T % 1024 == 0, "alignment");
};

// Place in the ring of KQS buffers and the parity of the round, of one chunk after another.
struct Ring {
    int s = 0;
    uint32_t par = 0;
    __device__ __forceinline__ void next()
    {
        if (++s == Layout::KQS) {
            s = 0;
            par ^= 1;
        }
    }
};

// An operand of a tf32 product, rounded to nearest.
__device__ __forceinline__ uint32_t tf32(float x)
{
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}

// Waits for a phase. The producer waits for every chunk's buffers in turn, with a limit, and sets the flag at shared
// address `flag` when one does not come back; the others wait until their phase comes or that flag is set, and go on all
// the same, so that every barrier keeps its count and the CTA comes to its end (a wait then lasts one poll): what they make
// is void, and the flag becomes an error. This keeps a wait short, which counts for the kernel's size.
__device__ __forceinline__ void wait_or_flag(uint32_t b, uint32_t par, uint32_t flag)
{
    if (!smem_ok(b, 8)) return;
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 f;\n"
                 "W%=:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1, %3;\n\t@p bra D%=;\n\t"
                 "ld.volatile.shared.u32 f, [%2];\n\tsetp.eq.u32 p, f, 0;\n\t@p bra W%=;\n"
                 "D%=:\n\t}" ::"r"(b),
                 "r"(par), "r"(flag), "r"(2000)  // ns that a poll may last
                 : "memory");
}

// log(1 + 2^(u log2 e)). Away from 0 by the hardware's logarithm, off by 2^-22; where e^u is below 1/32, whose logarithm of
// 1 + e^u would lose what it is there for, by the series, which leaves out e^4 / 5 of it, 2^-22. The few instructions count
// for the kernel's size. NaN comes through.
__device__ __forceinline__ float softplus_fast(float u)
{
    const float e = ex2_approx(-fabsf(u) * LOG2E), small = e * fmaf(e, fmaf(e, fmaf(e, -0.25f, 1.f / 3.f), -0.5f), 1.f);
    const float l = e < 0.03125f ? small : lg2_approx(1.f + e) * (1.f / LOG2E);
    return u > 0.f ? u + l : l;
}

// Rows of a sequence token by token: rows 8 g .. 8 g + 7 for every set bit of `groups`.
__device__ __noinline__ void walk_groups(const GdnParams &p, int seq, int h, const Span &sp, uint32_t groups)
{
    for (int g = threadIdx.x >> 5; g < DH / gdn::ROWS; g += NTHREADS / 32)
        if (groups >> g & 1) gdn::walk_rows(p, seq, h, sp, gdn::ROWS * g);
}

__global__ void __launch_bounds__(NTHREADS, 1)
    kda_gdn_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                      const __grid_constant__ CUtensorMap to, const __grid_constant__ GdnParams p)
{
    using Lay = Layout;
    extern __shared__ __align__(1024) uint8_t smem_dyn_tiles[];
    uint8_t *smem = smem_dyn_tiles;
    const uint32_t sb = smem_u32(smem);
#define SM_AT(T, a) (*reinterpret_cast<T *>(smem + (smem_checked((a), sizeof(T), sb) - sb)))
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % p.H, slot = blockIdx.x / p.H, hk = h / (p.H / p.HK);
    const int seq = p.cu && p.nseq <= LPT_MAX_SEQS ? ssmtc::longest_first(p, slot) : slot;
    if (p.cu && blockIdx.x == 0) blk::check_bounds(p.cu, p.nseq, p.total);
    Span sp = gdn::gdn_span(p, seq);
    if (!sp.ok) return;  // CTA-uniform, before any tensor memory is taken
    if (sp.len <= gdn::STEP_TOKENS) {  // as uniform; a packed call's short sequences are answered as they are alone
        if (!p.split) walk_groups(p, seq, h, sp, (1u << (DH / gdn::ROWS)) - 1u);
        return;
    }
    const int nch = (sp.len + C - 1) / C;

    volatile int *flags = reinterpret_cast<volatile int *>(smem + Lay::FLAGS);
    uint32_t *const spoilt = reinterpret_cast<uint32_t *>(smem + Lay::FLAGS) + 1;
    auto bar = [&](int i) { return sb + Lay::BAR + 8 * i; };
    auto kq = [&](const Ring &g) { return sb + Lay::KQ + g.s * Lay::KQT; };
    const uint32_t vt = sb + Lay::V;
    auto pt = [&](const Ring &g) { return sb + Lay::P + g.s * Lay::PT; };
    auto tt = [&](int n) { return sb + Lay::T + (n & 1) * Lay::BOX; };
    auto sc = [&](int n) { return sb + Lay::SC + (n & 3) * SC_BYTES; };
    auto live_of = [&](int n) { return min(C, sp.len - n * C); };

    if (warp == 0) {
        tc::alloc(sb + Lay::TMEMPTR, TMEM_COLS);
        tc::relinquish();
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < Lay::KQS; ++i) {
            mbar_init(bar(Lay::KQ_FULL + i), 1);
            mbar_init(bar(Lay::KQ_EMPTY + i), 2);
            mbar_init(bar(Lay::SC_FULL + i), 1);
            mbar_init(bar(Lay::T_FULL + i), 4);
            mbar_init(bar(Lay::FACT + i), 4);
        }
        for (int i : {Lay::V_FULL, Lay::V_EMPTY, Lay::G_DONE, Lay::G_DONE + 1, Lay::T_EMPTY, Lay::T_EMPTY + 1, Lay::D1_DONE, Lay::N_DONE, Lay::S_DONE, Lay::O_DONE, Lay::SQ_DONE, Lay::U_DONE, Lay::END, Lay::END2, Lay::END3})
            mbar_init(bar(i), 1);
        mbar_init(bar(Lay::KQ_ZERO), 4);
        mbar_init(bar(Lay::OUT_RD), 4);
        mbar_init(bar(Lay::KQ_FREE), 4);
        for (int i : {Lay::SB_GO, Lay::D1_GO, Lay::N_GO}) mbar_init(bar(i), 8);
        flags[0] = 0;
        *spoilt = 0u;
        fence_mbar_init();
    }
    // the parts of T above its diagonal blocks are zero for good
    for (int i = threadIdx.x; i < Lay::TS * Lay::BOX / 16; i += NTHREADS) SM_AT(uint4, sb + Lay::T + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_async_smem();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    // the allocation is the whole tensor memory, so it starts at address 0
    constexpr uint32_t tmem = 0;
    if ((*reinterpret_cast<volatile uint32_t *>(smem + Lay::TMEMPTR) != tmem || (sb & 1023u)) && threadIdx.x == 0) flags[0] = 1;
    const uint32_t flag = sb + Lay::FLAGS;
    auto wait_w = [&](int b, uint32_t par) {
        wait_or_flag(bar(b), par, flag);
        __syncwarp();
    };
    auto arrive_w = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b));
    };
    // operands: K step i of a K-major [K; Q] tile, of an MN-major tile (16 rows), of a tile of 128-byte rows, of one of fp32, and
    // of an operand in tensor memory that two warps have written halves of
    constexpr uint32_t HI = tc::sdesc_hi(1024, tc::SWZ_128B);
    constexpr uint32_t id_n = tc::idesc(tc::BF16, 128, C, 0, 0), id_u = tc::idesc(tc::BF16, 128, C, 1, 0), id_s = tc::idesc(tc::BF16, 128, DH, 0, 1),
                       id_o = tc::idesc(tc::TF32, 128, C, 0, 0);
    auto kmaj = [](uint32_t lo, int i) { return tc::sdesc_of<HI>(lo + static_cast<uint32_t>(((i >> 2) * 2 * Lay::BOX + (i & 3) * 32) >> 4)); };
    auto nmaj = [](uint32_t lo, int i) { return tc::sdesc_of<HI>(lo + static_cast<uint32_t>((i * 16 * 128) >> 4)); };
    auto rows = [](uint32_t lo, int i) { return tc::sdesc_of<HI>(lo + static_cast<uint32_t>((i * 32) >> 4)); };
    auto rows32 = [](uint32_t lo, int i) { return tc::sdesc_of<HI>(lo + static_cast<uint32_t>(((i >> 2) * Lay::BOX + (i & 3) * 32) >> 4)); };
    auto halves = [](int i) { return static_cast<uint32_t>(32 * (i >> 1) + 8 * (i & 1)); };
    // a [K; Q] tile is there, with the rows past the sequence's end cleared
    auto wait_kq = [&](int n, const Ring &g) {
        wait_w(Lay::KQ_FULL + g.s, g.par);
        if (live_of(n) < C) wait_w(Lay::KQ_ZERO, 0);
    };
    // the products of an issuer that are still on their way when its loop is left
    auto finish = [&](int b) {
        tc::commit_w(bar(b));
        if (lane == 0) drain_bar(bar(b), 0);
        __syncwarp();
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        if (lane == 0) {
            tma_prefetch_desc(&tq);
            tma_prefetch_desc(&tk);
            tma_prefetch_desc(&tv);
            Ring rg;
            int nk = 0, nv = 0;  // tiles issued
#pragma unroll 1
            for (int n = 0; n <= nch; ++n, rg.next()) {
                if (n < nch) {
                    const int tok = sp.bos + n * C, full = Lay::KQ_FULL + rg.s;
                    if (!wait_bar(bar(Lay::KQ_EMPTY + rg.s), rg.par ^ 1, flags)) break;
                    mbar_arrive_expect_tx(bar(full), Lay::KQT);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tma_load_3d(kq(rg) + 2 * c * Lay::BOX, &tk, 64 * c, hk, tok, bar(full));
                        tma_load_3d(kq(rg) + (2 * c + 1) * Lay::BOX, &tq, 64 * c, hk, tok, bar(full));
                    }
                    ++nk;
                    // a tile's buffer is free late, so the next ones are on their way to L2 by then
                    if (n + Lay::KQS < nch) {
                        const int ahead = tok + Lay::KQS * C;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            tma_prefetch_3d(&tk, 64 * c, hk, ahead);
                            tma_prefetch_3d(&tq, 64 * c, hk, ahead);
                            tma_prefetch_3d(&tv, 64 * c, h, ahead);
                        }
                    }
                }
                // V's one buffer is free when the last V has met its T, most of a chunk before this one is wanted
                if (n > 0) {
                    if (!wait_bar(bar(Lay::V_EMPTY), n & 1, flags)) break;
                    mbar_arrive_expect_tx(bar(Lay::V_FULL), Lay::VT);
#pragma unroll
                    for (int c = 0; c < 2; ++c) tma_load_3d(vt + c * Lay::BOX, &tv, 64 * c, h, sp.bos + (n - 1) * C, bar(Lay::V_FULL));
                    ++nv;
                }
            }
            // no copy is in flight when the CTA ends, whichever way the loop was left
            for (int m = max(nk - Lay::KQS, 0); m < nk; ++m) drain_bar(bar(Lay::KQ_FULL + m % Lay::KQS), (m / Lay::KQS) & 1);
            if (nv > 0) drain_bar(bar(Lay::V_FULL), (nv - 1) & 1);
            // and the watch over the others' waits lasts until the last chunk's output
            for (int m = max(nk - Lay::KQS, 0); m < nk; ++m) wait_bar(bar(Lay::KQ_EMPTY + m % Lay::KQS), (m / Lay::KQS) & 1, flags);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer: chain (whole warp)
        Ring rg;
#pragma unroll 1
        for (int n = 0; n < nch; ++n, rg.next()) {
            const uint32_t dk = tc::sdesc_lo(kq(rg), 16), dt = tc::sdesc_lo(tt(n), 16), dkn = tc::sdesc_lo(kq(rg), 2 * Lay::BOX);
            wait_kq(n, rg);
            wait_w(Lay::SB_GO, n & 1);
            tc::fence_after();
#pragma unroll 1
            for (int i = 0; i < 8; ++i) tc::mma_ts_w(tmem + T_D1, tmem + T_SB + 8 * i, kmaj(dk, i), id_n, i > 0);
            tc::commit_w(bar(Lay::D1_DONE));
            wait_w(Lay::U_DONE, n & 1);
            wait_w(Lay::D1_GO, n & 1);
            tc::fence_after();
#pragma unroll 1
            for (int i = 0; i < 4; ++i)  // outputs from 16 i on: rows of T by 2048 bytes, columns of D2, N by 16
                tc::mma_ts_w(tmem + T_D2 + 16 * i, tmem + T_D1 + halves(i), rows(dt + 128 * i, i), id_n - (i << 18), 1);
            tc::commit_w(bar(Lay::N_DONE));
            tc::commit_w(bar(Lay::T_EMPTY + (n & 1)));
            // (with the product of this state and Q done, S_DONE frees its copy too)
            wait_w(Lay::SQ_DONE, n & 1);
            wait_w(Lay::N_GO, n & 1);
            tc::fence_after();
#pragma unroll 1
            for (int i = 0; i < 4; ++i) tc::mma_ts_w(tmem + T_S, tmem + T_D1 + halves(i), nmaj(dkn, i), id_s, 1);
            tc::commit_w(bar(Lay::S_DONE));
            tc::commit_w(bar(Lay::KQ_EMPTY + rg.s));
        }
        finish(Lay::END);
    } else if (warp == 2) {
        // ---------------------------------------------------------------- MMA issuer: [K; Q] K^T, V^T T^T
        auto issue_g = [&](int n, const Ring &rg) {
            wait_kq(n, rg);
            if (n > 0) wait_w(Lay::KQ_FREE, (n - 1) & 1);
            tc::fence_after();
            const uint32_t d = tc::sdesc_lo(kq(rg), 16);
#pragma unroll 1
            for (int i = 0; i < 8; ++i) tc::mma_ss_w(tmem + T_KQ, kmaj(d, i), kmaj(d, i), id_n, i > 0);
            tc::commit_w(bar(Lay::G_DONE + (n & 1)));  // either group sees every phase of its own
        };
        auto issue_u = [&](int n, const Ring &rg) {
            wait_w(Lay::V_FULL, n & 1);
            if (const int Lv = live_of(n); Lv < C) {  // as the rows of K and Q past the end, which other warps clear
                for (int i = lane; i < (C - Lv) * 16; i += 32) {
                    const int r = Lv + (i >> 4), c = i & 15;
                    SM_AT(uint4, vt + (c >> 3) * Lay::BOX + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                tc::fence_async_smem();
                __syncwarp();
            }
            // the last chunk's N, whose columns these are, has been multiplied, and N' made of it
            if (n > 0) {
                wait_w(Lay::O_DONE, (n - 1) & 1);
                wait_w(Lay::S_DONE, (n - 1) & 1);
            }
            wait_w(Lay::T_FULL + rg.s, rg.par);
            tc::fence_after();
            const uint32_t dv = tc::sdesc_lo(vt, Lay::BOX), dt = tc::sdesc_lo(tt(n), 16);
#pragma unroll 1
            for (int i = 0; i < 4; ++i) tc::mma_ss_w(tmem + T_D2, nmaj(dv, i), rows(dt, i), id_u, i > 0);
            tc::commit_w(bar(Lay::U_DONE));
            tc::commit_w(bar(Lay::V_EMPTY));
        };
        Ring rg, ru;
#pragma unroll 1
        for (int n = 0; n <= nch; ++n) {  // one chunk ahead with the first
            if (n < nch) issue_g(n, rg);
            rg.next();
            if (n == 0) continue;
            issue_u(n - 1, ru);
            ru.next();
        }
        finish(Lay::END2);
    } else if (warp == 3) {
        // ---------------------------------------------------------------- decays and steps, two tokens per lane; output MMAs
        Ring rg;
        const float A2 = -expf(__ldg(p.A_log + h)) * LOG2E, bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f;
        const uint16_t *ap = p.a + static_cast<long long>(sp.bos) * p.as + h, *bp = p.beta + static_cast<long long>(sp.bos) * p.bs + h;
        uint32_t ra[2] = {0u, 0u}, rb[2] = {0u, 0u};
        auto fetch = [&](int n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = n * C + 2 * lane + i;
                if (t < sp.len) {
                    ra[i] = ap[t * p.as];
                    rb[i] = bp[t * p.bs];
                }
            }
        };
        fetch(0);
        Ring rs;  // of the scalars, three chunks ahead
#pragma unroll 1
        for (int n = -Lay::KQS; n < nch; ++n) {
            if (n >= 0) {
                const uint32_t dq = tc::sdesc_lo(kq(rg), 16) + (Lay::BOX >> 4), dp = tc::sdesc_lo(pt(rg), 16);
                wait_kq(n, rg);
                if (n > 0) wait_w(Lay::OUT_RD, (n - 1) & 1);
                wait_w(Lay::SB_GO, n & 1);
                tc::fence_after();
#pragma unroll 1
                for (int i = 0; i < 8; ++i) tc::mma_ts_w(tmem + T_SQ, tmem + T_SB + 8 * i, kmaj(dq, i), id_n, i > 0);
                tc::commit_w(bar(Lay::SQ_DONE));
                wait_w(Lay::T_FULL + rg.s, rg.par);
                wait_w(Lay::N_DONE, n & 1);
                tc::fence_after();
#pragma unroll 1
                for (int i = 0; i < 8; ++i)  // eight tokens j, outputs as above
                    tc::mma_ts_tf32_w(tmem + T_PV + 16 * (i >> 1), tmem + T_D2 + 8 * i, rows32(dp + 128 * (i >> 1), i), id_o - ((i >> 1) << 18), i > 0);
                tc::commit_w(bar(Lay::O_DONE));
                tc::commit_w(bar(Lay::KQ_EMPTY + rg.s));
                rg.next();
            }
            if (const int m = n + Lay::KQS; m < nch) {
                const int Lv = live_of(m);
                float a[2], b[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool live = 2 * lane + i < Lv;
                    // held at the least decay by a comparison that lets NaN through (fmaxf would not)
                    const float u = A2 * softplus_fast(__uint_as_float(ra[i] << 16) + bias);
                    a[i] = !live ? 0.f : u < ssm::MIN_LOG2_DECAY ? ssm::MIN_LOG2_DECAY : u;
                    b[i] = live ? blk::sigmoid_fast(__uint_as_float(rb[i] << 16)) : 0.f;
                }
                fetch(m + 1);
                float pre = a[0] + a[1];
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const float u = __shfl_up_sync(0xffffffffu, pre, d);
                    if (lane >= d) pre += u;
                }
                const float all = __shfl_sync(0xffffffffu, pre, 31);
                const float g1 = pre, before = __shfl_up_sync(0xffffffffu, pre, 1), g0 = (lane ? before : 0.f) + a[0];
                wait_w(Lay::KQ_EMPTY + rs.s, rs.par ^ 1);  // its buffer is free with that of the tile three chunks back
                const uint32_t o = sc(m) + 8 * lane;
                SM_AT(float2, o + SC_G) = make_float2(g0, g1);
                SM_AT(float2, o + SC_B) = make_float2(b[0], b[1]);
                SM_AT(float2, o + SC_D) = make_float2(ex2_approx(g0), ex2_approx(g1));
                SM_AT(float2, o + SC_N) = make_float2(ex2_approx(all - g0), ex2_approx(all - g1));
                if (lane == 0) SM_AT(float, sc(m) + SC_GAM) = ex2_approx(all);
                arrive_w(Lay::SC_FULL + rs.s);
                rs.next();
            }
        }
        finish(Lay::END3);
    } else if (warp < 12) {
        // ---------------------------------------------------------------- chain
        Ring rg;
        const int q = warp & 3, hf = warp < 8 ? 0 : 1, v = 32 * q + lane;
        const uint32_t lq = tmem + (static_cast<uint32_t>(32 * q) << 16);
        const uint32_t ls = lq + T_S + 64 * hf, lsb = lq + T_SB + 32 * hf, l1 = lq + T_D1 + 32 * hf, l2 = lq + T_D2 + 32 * hf;
        const size_t row = ((static_cast<size_t>(seq) * p.H + h) * DH + v) * DH + 64 * hf;  // of this thread's part of the state
        auto load_init = [&](int c, uint32_t(&r)[32]) {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0u;
            if (!p.init || !gmem_ok(row + c, 32, gdn::state_elems(p))) return;
            if (p.init_dtype == KDA_DTYPE_FP32) {
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const float *>(p.init) + row + c + i);
                    r[i] = w.x; r[i + 1] = w.y; r[i + 2] = w.z; r[i + 3] = w.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.init) + row + c + i);
                    r[i] = w.x << 16; r[i + 1] = w.x & 0xffff0000u; r[i + 2] = w.y << 16; r[i + 3] = w.y & 0xffff0000u;
                    r[i + 4] = w.z << 16; r[i + 5] = w.z & 0xffff0000u; r[i + 6] = w.w << 16; r[i + 7] = w.w & 0xffff0000u;
                }
            }
        };
        auto store_fin = [&](int c, const uint32_t(&r)[32]) {
            if (!gmem_ok(row + c, 32, gdn::state_elems(p))) return;
            if (p.fin_dtype == KDA_DTYPE_FP32) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<uint4 *>(static_cast<float *>(p.fin) + row + c + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    auto two = [&](int j) { return pack_bf16(__uint_as_float(r[i + j]), __uint_as_float(r[i + j + 1])); };
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.fin) + row + c + i) = make_uint4(two(0), two(2), two(4), two(6));
                }
            }
        };
        // 16 columns as 8 of an operand, as they are or times the factors at `at`
        auto pack = [](const uint32_t(&r)[16], uint32_t(&o)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        };
        auto pack_scaled = [&](const uint32_t(&r)[16], uint32_t(&o)[8], uint32_t at) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 f = SM_AT(const float4, at + 4 * i);
                const float2 x = fmul2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), make_float2(f.x, f.y));
                const float2 y = fmul2(make_float2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), make_float2(f.z, f.w));
                o[i / 2] = pack_bf16(x.x, x.y);
                o[i / 2 + 1] = pack_bf16(y.x, y.y);
            }
        };
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
            uint32_t r[32];
            load_init(32 * g, r);
            __syncwarp();
            tc::st32(ls + 32 * g, r);
        }
        tc::wait_st();
        // Loops are left rolled here and below: the roles' code together is larger than the instruction caches next to the
        // schedulers, and what is fetched twice costs more than a branch.
#pragma unroll 1
        for (int n = 0; n < nch; ++n, rg.next()) {
            uint32_t r[16], o[8];
            // the state as an operand
            if (n > 0) wait_w(Lay::S_DONE, (n - 1) & 1);
            tc::fence_after();
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                tc::ld16(ls + 16 * g, r);
                tc::wait_ld();
                pack(r, o);
                tc::st8(lsb + 8 * g, o);
            }
            tc::wait_st();
            tc::fence_before();
            arrive_w(Lay::SB_GO);
            // decayed in place
            wait_w(Lay::SC_FULL + rg.s, rg.par);
            const float gam = SM_AT(const float, sc(n) + SC_GAM);
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                tc::ld16(ls + 16 * g, r);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 x = fmul2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), make_float2(gam, gam));
                    r[i] = __float_as_uint(x.x);
                    r[i + 1] = __float_as_uint(x.y);
                }
                tc::st16(ls + 16 * g, r);
            }
            // D1' over D1
            wait_w(Lay::D1_DONE, n & 1);
            wait_w(Lay::T_FULL + rg.s, rg.par);
            tc::fence_after();
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
                tc::ld16(l1 + 16 * g, r);
                tc::wait_ld();
                pack_scaled(r, o, sc(n) + SC_D + 128 * hf + 64 * g);
                tc::st8(l1 + 8 * g, o);
            }
            tc::wait_st();
            tc::fence_before();
            arrive_w(Lay::D1_GO);
            // N' of N, over D1'
            wait_w(Lay::N_DONE, n & 1);
            tc::fence_after();
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
                tc::ld16(l2 + 16 * g, r);
                tc::wait_ld();
                pack_scaled(r, o, sc(n) + SC_N + 128 * hf + 64 * g);
                tc::st8(l1 + 8 * g, o);
            }
            tc::wait_st();
            tc::fence_before();
            arrive_w(Lay::N_GO);
        }
        wait_w(Lay::S_DONE, (nch - 1) & 1);
        tc::fence_after();
        float2 z = make_float2(0.f, 0.f);  // 0 NaN and 0 inf are NaN
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
            uint32_t r[32];
            tc::ld32(ls + 32 * g, r);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 2) z = ffma2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), make_float2(0.f, 0.f), z);
        }
        if (!(z.x + z.y == 0.f)) atomicOr(spoilt, 1u << (v / gdn::ROWS));
        named_bar_sync(4 + q, 64);  // both halves of these rows have been looked at
        if (p.fin) {
            const bool number = !(*const_cast<volatile uint32_t *>(spoilt) >> (v / gdn::ROWS) & 1u);  // else made again at the end
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
                uint32_t r[32];
                tc::ld32(ls + 32 * g, r);  // every lane of the warp takes part in the load
                tc::wait_ld();
                if (number) store_fin(32 * g, r);
                __syncwarp();
            }
        }
        tc::fence_before();
    } else if (warp < 16) {
        // ---------------------------------------------------------------- output
        Ring rg;
        const int q = warp & 3;
        const uint32_t lq = tmem + (static_cast<uint32_t>(32 * q) << 16);
        // The factors of rows and columns of a chunk, a row of K or Q per thread, two chunks ahead
        auto factors = [&](int n, const Ring &g) {
            wait_w(Lay::KQ_FULL + g.s, g.par);
            wait_w(Lay::SC_FULL + g.s, g.par);
            const int Lv = live_of(n), r = 32 * (q & 1) + lane;
            const bool is_q = q >= 2;
            const uint32_t s = sc(n) + 4 * r, at = kq(g) + (is_q ? Lay::BOX : 0) + r * 128;
            auto vec = [&](int c) { return at + (c >> 3) * 2 * Lay::BOX + (((c & 7) ^ (r & 7)) << 4); };
            if (Lv < C) {
                // rows past the end hold another sequence's tokens: zero, so that a NaN there meets no product
                if (r >= Lv)
#pragma unroll 1
                    for (int c = 0; c < 16; ++c) SM_AT(uint4, vec(c)) = make_uint4(0u, 0u, 0u, 0u);
                tc::fence_async_smem();
                arrive_w(Lay::KQ_ZERO);
            }
            float f = 1.f;
            if (p.l2) {
                float2 ss = make_float2(0.f, 0.f);
#pragma unroll 4
                for (int c = 0; c < 16; ++c) {
                    float2 x[4];
                    blk::unpack8(SM_AT(const uint4, vec(c)), x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) ss = ffma2(x[j], x[j], ss);
                }
                f = rsqrtf(ss.x + ss.y + gdn::L2_EPS);
            }
            const float G = SM_AT(const float, s + SC_G);
            if (is_q) {
                f *= p.scale;
                SM_AT(float, s + SC_FQ) = f;
                SM_AT(float, s + SC_O) = f * ex2_approx(G);
            } else {
                const float b = SM_AT(const float, s + SC_B), fd = SM_AT(const float, s + SC_D), fn = SM_AT(const float, s + SC_N);
                SM_AT(float, s + SC_FK) = f;
                SM_AT(float, s + SC_GK) = G - lg2_approx(f * b);  // b = 0: infinity, and the factor is 0
                SM_AT(float, s + SC_D) = -fd * f;
                SM_AT(float, s + SC_N) = fn * f * b;
            }
            arrive_w(Lay::FACT + g.s);
        };
        Ring ra;
#pragma unroll 1
        for (int n = -2; n < nch; ++n) {
            if (n + 2 < nch) factors(n + 2, ra);
            ra.next();
            if (n < 0) continue;
            const int Lv = live_of(n);
            if (warp == 12) {
                if (lane == 0) bulk_wait_read();  // the last chunk's store is done with the buffer
                __syncwarp();
            }
            wait_w(Lay::T_FULL + rg.s, rg.par);
            wait_w(Lay::O_DONE, n & 1);
            named_bar_sync(1, 128);
            tc::fence_after();
            // The accumulators are loaded as warp MMA fragments (8 channels x 8 tokens), so that stmatrix.trans hands a token's
            // row its 16 bytes of eight channels.
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {  // 16 channels x 32 tokens
                const int lh = g >> 1, c0 = 32 * (g & 1);
                const uint32_t la = lq + (static_cast<uint32_t>(16 * lh) << 16) + c0;
                uint32_t s[16], u[16], o[8];
                tc::ld_16x256b_x4(la + T_SQ, s);
                tc::ld_16x256b_x4(la + T_PV, u);
                float2 f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = SM_AT(const float2, sc(n) + SC_O + 4 * (c0 + 8 * i + 2 * (lane & 3)));
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 y = ffma2(f[i >> 1], make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])),
                                           make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])));
                    o[i] = pack_bf16(y.x, y.y);
                }
                const int v8 = 4 * q + 2 * lh + ((lane >> 3) & 1), r = lane & 7;  // eight channels and token row of this lane's address
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = c0 + 16 * i + 8 * (lane >> 4) + r;
                    stsm_x4_t(sb + Lay::OUT + (v8 >> 3) * Lay::BOX + t * 128 + (((v8 & 7) ^ r) << 4), o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            tc::fence_before();
            arrive_w(Lay::OUT_RD);
            tc::fence_async_smem();
            named_bar_sync(1, 128);
            if (Lv == C) {
                if (warp == 12 && lane == 0) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) tma_store_3d(&to, sb + Lay::OUT + c * Lay::BOX, 64 * c, h, sp.bos + n * C);
                    bulk_commit();
                }
            } else {
                for (int i = threadIdx.x - 384; i < Lv * 16; i += 128) {
                    const int t = i >> 4, g = i & 15;
                    const long long e = static_cast<long long>(sp.bos + n * C + t) * p.os + static_cast<long long>(h) * DH + 8 * g;
                    if (!gmem_ok(e, 8, (p.total - 1) * p.os + static_cast<long long>(p.H) * DH)) continue;
                    *reinterpret_cast<uint4 *>(p.out + e) =
                        SM_AT(const uint4, sb + Lay::OUT + (g >> 3) * Lay::BOX + t * 128 + (((g & 7) ^ (t & 7)) << 4));
                }
            }
            rg.next();
        }
        if (warp == 12 && lane == 0) bulk_wait_all();
    } else {
        // ---------------------------------------------------------------- A, P and T
        Ring rg;
        // Two groups of four warps take turns. Quarters 0 and 1 of tensor memory hold K K^T, 2 and 3 Q K^T.
        const int q = warp & 3, grp = (warp - 16) >> 2;
        const int lo = q & 1, i0 = 32 * lo + lane;  // this thread's row
        const uint32_t lq = tmem + (static_cast<uint32_t>(32 * q) << 16) + T_KQ;
        const uint32_t scr = sb + Lay::SCR + grp * Lay::SCRATCH;
        auto bits = [](float x) { return __float_as_uint(x); };
        auto at = [&](int i, int j) { return scr + 4 * ((i < 32 ? i * Lay::LD0 : 32 * Lay::LD0 + (i - 32) * Lay::LD1) + j); };
        auto A = [&](int i, int j) -> float & { return SM_AT(float, at(i, j)); };
        auto sync = [&] { named_bar_sync(2 + grp, 128); };
        const int g8 = lane >> 2, t4 = lane & 3;
        // d += X[xr.., xc..] Y[yr.., yc..], 16 x 16 by 16 x 8, both in the scratch. What is not A itself is rounded to tf32
        // as it is put there; A is cut off, by 2^-11 of it in the mean.
        auto product = [&](float(&d)[4], int xr, int xc, int yr, int yc) {
            const uint32_t x = at(xr + g8, xc + t4), xd = 32 * (xr < 32 ? Lay::LD0 : Lay::LD1), y = at(yr + t4, yc + g8), yd = 16 * (yr < 32 ? Lay::LD0 : Lay::LD1);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t a[4] = {SM_AT(uint32_t, x + 32 * k), SM_AT(uint32_t, x + xd + 32 * k), SM_AT(uint32_t, x + 32 * k + 16), SM_AT(uint32_t, x + xd + 32 * k + 16)};
                mma_tf32(d, a, SM_AT(uint32_t, y + 2 * k * yd), SM_AT(uint32_t, y + (2 * k + 1) * yd));
            }
        };
        auto put = [&](const float(&d)[4], int r, int c, float f) {
            SM_AT(uint2, at(r + g8, c + 2 * t4)) = make_uint2(tf32(f * d[0]), tf32(f * d[1]));
            SM_AT(uint2, at(r + g8 + 8, c + 2 * t4)) = make_uint2(tf32(f * d[2]), tf32(f * d[3]));
        };
        if (grp) rg.next();
#pragma unroll 1
        for (int n = grp; n < nch; n += 2) {
            const uint32_t s = sc(n), t0 = tt(n);
            // where T[i][j] stands as an operand
            auto t_at = [&](int i, int j) { return t0 + i * 128 + (((j >> 3) ^ (i & 7)) << 4) + (j & 7) * 2; };
            auto put_t = [&](const float(&d)[4], int r, int c) {
                SM_AT(uint32_t, t_at(r + g8, c + 2 * t4)) = pack_bf16(-d[0], -d[1]);
                SM_AT(uint32_t, t_at(r + g8 + 8, c + 2 * t4)) = pack_bf16(-d[2], -d[3]);
            };
            wait_w(Lay::FACT + rg.s, rg.par);
            const float Gi = SM_AT(const float, s + SC_G + 4 * i0), fi = SM_AT(const float, s + (q < 2 ? SC_FK : SC_FQ) + 4 * i0);
            wait_w(Lay::G_DONE + (n & 1), (n >> 1) & 1);
            tc::fence_after();
            // A and P up to their diagonal, 16 columns at a time
#pragma unroll 1
            for (int b = 0; b < 32 * (lo + 1); b += 16) {
                uint32_t r[16];
                float2 w[8];
                tc::ld16(lq + b, r);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float4 g = SM_AT(const float4, s + SC_GK + 4 * (b + 2 * j));
                    w[j] = make_float2(ex2_approx(Gi - g.x), ex2_approx(Gi - g.y));
                    w[j + 1] = make_float2(ex2_approx(Gi - g.z), ex2_approx(Gi - g.w));
                }
                tc::wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = fmul2(fmul2(w[j], make_float2(fi, fi)), make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])));
                if (q < 2) {
                    // of what is not below the diagonal, only the upper right 8 x 8 of a diagonal block is read: zero
                    const bool off = (i0 & ~7) == b;
#pragma unroll
                    for (int j = 4; j < 8; ++j) w[j] = off ? make_float2(0.f, 0.f) : w[j];
#pragma unroll
                    for (int j = 0; j < 8; j += 2) SM_AT(float4, at(i0, b + 2 * j)) = make_float4(w[j].x, w[j].y, w[j + 1].x, w[j + 1].y);
                } else {
                    if (b >= 32 * lo) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (b + 2 * j > i0) w[j].x = 0.f;
                            if (b + 2 * j + 1 > i0) w[j].y = 0.f;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; j += 2)
                        SM_AT(float4, pt(rg) + (b >> 5) * Lay::BOX + i0 * 128 + ((((b >> 2 & 4) + (j >> 1)) ^ (i0 & 7)) << 4)) = make_float4(w[j].x, w[j].y, w[j + 1].x, w[j + 1].y);
                }
            }
            tc::fence_before();
            arrive_w(Lay::KQ_FREE);
            sync();
            wait_w(Lay::T_EMPTY + (n & 1), ((n >> 1) & 1) ^ 1);  // T's buffer has been read up two chunks back
            // (I + A)^-1: diagonal blocks of 8, two per warp, a row per lane; then the block between them
            {
                const int d0 = 16 * q, d1 = d0 + (lane & 8), c = lane & 7;
                // row c of the inverse, x (I + A) = e_c, from its last column to its first
                const uint32_t ad = at(d1, d1), ld = 4 * (q < 2 ? Lay::LD0 : Lay::LD1);
                float x[8];
#pragma unroll
                for (int j = 7; j >= 0; --j) {
                    float u = j == c ? 1.f : 0.f, w = 0.f;
#pragma unroll
                    for (int i = j + 1; i < 8; ++i)
                        if ((i - j) & 1)
                            u = fmaf(-SM_AT(const float, ad + i * ld + 4 * j), x[i], u);
                        else
                            w = fmaf(-SM_AT(const float, ad + i * ld + 4 * j), x[i], w);
                    x[j] = u + w;
                }
                __syncwarp();
                if (lane < 16) {
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        SM_AT(uint4, at(d1 + c, d1 + j)) = make_uint4(tf32(x[j]), tf32(x[j + 1]), tf32(x[j + 2]), tf32(x[j + 3]));
                        o[j / 2] = pack_bf16(x[j], x[j + 1]);
                        o[j / 2 + 1] = pack_bf16(x[j + 2], x[j + 3]);
                    }
                    SM_AT(uint4, t_at(d1 + c, d1)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                __syncwarp();
                float d[4] = {}, e[4] = {};
                const uint32_t a[4] = {bits(A(d0 + 8 + g8, d0 + t4)), 0u, bits(A(d0 + 8 + g8, d0 + t4 + 4)), 0u};
                mma_tf32(d, a, bits(A(d0 + t4, d0 + g8)), bits(A(d0 + t4 + 4, d0 + g8)));
                __syncwarp();
                SM_AT(uint2, at(d0 + 8 + g8, d0 + 2 * t4)) = make_uint2(tf32(d[0]), tf32(d[1]));
                __syncwarp();
                const uint32_t h[4] = {bits(A(d0 + 8 + g8, d0 + 8 + t4)), 0u, bits(A(d0 + 8 + g8, d0 + 8 + t4 + 4)), 0u};
                mma_tf32(e, h, bits(A(d0 + 8 + t4, d0 + g8)), bits(A(d0 + 8 + t4 + 4, d0 + g8)));
                __syncwarp();
                SM_AT(uint2, at(d0 + 8 + g8, d0 + 2 * t4)) = make_uint2(tf32(-e[0]), tf32(-e[1]));
                SM_AT(uint32_t, t_at(d0 + 8 + g8, d0 + 2 * t4)) = pack_bf16(-e[0], -e[1]);
            }
            sync();
            // the blocks below: -T_hi A_hl T_lo, first of 16 (eight columns per warp), then of 32
            {
                const int c0 = 32 * (q & 1), r0 = c0 + 16, n8 = 8 * (q >> 1);
                float d[4] = {}, e[4] = {};
                product(d, r0, c0, c0, c0 + n8);
                put(d, c0, r0 + n8, 1.f);  // above the diagonal, where nothing stands
                __syncwarp();
                product(e, r0, r0, c0, r0 + n8);
                __syncwarp();
                put(e, c0, r0 + n8, -1.f);  // there too: the other warp may still read A
                put_t(e, r0, c0 + n8);
            }
            sync();
            {
                const int mi = 16 * (q >> 1), n0 = 8 * (q & 1);  // columns n0 .. and n0 + 16 ..
                float d[2][4] = {}, e[2][4] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    for (int k = 16 * h; k < 32; k += 16) {
                        const bool below = k > 16 * h;  // the block below the diagonal ones stands above them
                        product(d[h], 32 + mi, k, below ? 0 : k, below ? 16 + n0 : n0 + 16 * h);
                    }
                sync();
#pragma unroll
                for (int h = 0; h < 2; ++h) put(d[h], 32 + mi, n0 + 16 * h, 1.f);  // over A, which has been read
                sync();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    for (int k = 0; k <= mi; k += 16) {
                        const bool below = k < mi;
                        product(e[h], below ? 32 : 32 + mi, below ? 48 : 32 + k, 32 + k, n0 + 16 * h);
                    }
                    put_t(e[h], 32 + mi, n0 + 16 * h);
                }
            }
            tc::fence_async_smem();
            arrive_w(Lay::T_FULL + rg.s);
            rg.next();
            rg.next();
        }
    }

    tc::fence_before();
    __syncthreads();
    if (*flags && threadIdx.x == 0) atomicOr(&g_dev_error, DEVERR_TIMEOUT);
    const uint32_t groups = *spoilt;
    if (groups) walk_groups(p, seq, h, sp, groups);
    if (warp == 0) {
        __syncwarp();
        tc::fence_after();
        tc::dealloc(tmem, TMEM_COLS);
    }
#undef SM_AT
}

}  // namespace gdntc
}  // namespace kda
