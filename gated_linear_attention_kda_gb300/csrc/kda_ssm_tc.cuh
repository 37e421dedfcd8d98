// kda_ssm_tc.cuh -- the selective state-space scan over prompts on the 5th-generation tensor core,
// 128 tokens at a time.
//
// Chunk algebra. With a_t = -exp(A_log) delta_t, the recurrence S <- exp(a) S + delta x b^T,
// out = S c + D x over a chunk of tokens j = 0..127 that starts from S0 is
//   G[i, j] = c_i . b_j                                                    (per group)
//   M[i, j] = G[i, j] delta_j exp(a_{j+1} + ... + a_i)        for j <= i, else 0
//   out_i   = sum_j M[i, j] x_j + exp(a_0 + ... + a_i) S0 c_i + D x_i
//   S1      = exp(a_0 + ... + a_127) S0 + sum_j w_j x_j b_j^T,   w_j = delta_j exp(a_{j+1} + ... + a_127)
// Every exponent is a sum of terms of one sign taken directly: a chunk is four blocks of 32 tokens;
// between blocks the decay is the product of 2^(sum to the end of j's block) and 2^(sum from there to
// i), each at most 1, and only inside a block are two running sums subtracted (at most 32 terms, each
// held at or above -160). So nothing overflows, and the score matrix costs one exponential per token
// and block instead of one per entry away from the diagonal blocks.
//
// One CTA owns the state of one (sequence, head), or of one piece of its time axis, and walks its
// chunks. The state lives in tensor memory, fp32, transposed (lane = state channel n, column = head
// channel p), so that
//   G  [128 x 128] = C B^T               both straight from their TMA tiles (K-major)
//   Y  [128 x P]   = C S0^T              S0 rounded to bf16 in shared memory; rows then scaled in place
//   Y             += M X                 scores bf16 in tensor memory, X straight from its tile
//   S             += (w B)^T X           w B as bf16 parts in tensor memory, transposed on the way
// and D X is added to Y in fp32 as the rows are written.
// Roundings: M and S0 to bf16 as operands (the output is bf16; the carried state itself is not rounded);
// w B into PARTS bf16 parts of 8 bits each: 3, exact, where an fp32 state is returned, 2 (2^-17 of a term)
// where it is returned in bf16 or not at all. D is not rounded: on the diagonal of M it would lose sixteen
// bits, by the same error for every token of a head, and a score that is small against D most of its own
// (8 x 4096 tokens of 16 heads of 128 would take 96 us instead of 104, 16 packed prompts of 32 heads of 64
// 269 instead of 288; the outputs' relative error would be 2.36e-3 instead of 2.10e-3, of which 1.66e-3 are
// their own rounding). Sums are fp32.
//
// NaN: a product multiplies what the mask leaves out by zero, and 0 NaN is NaN, so a NaN or infinity in x (which is
// an MMA operand as it stands) reaches its channel's outputs of the whole chunk. It also leaves no number in that
// channel's state up to the end of the piece, where such channels show without a look at x. Their outputs ahead of the
// first such x in its chunk are then made again in fp32 (finish_spoilt): only calls that hold such an x pay for it
// (8 x 4096 tokens of 16 heads of 128, one NaN near the end of every sequence and head: 0.76 ms; in every channel
// 2.1 ms). A scan of each x tile would cost every call 14 to 19 %. In dt, b and c, which the warps handle, NaN reaches
// later tokens alone.
//
// What bounds it: 8 x 4096 tokens of 16 heads of 128 take 104 us (2.8 TB/s of HBM; 128 of the 152 SMs have a
// state), about 6,300 cycles a chunk. Of these the MMAs take 3,072 (1,536 of them for the three parts of w B)
// and shared memory 4,096: the MMAs read 256 KB of operands, TMA moves 128 KB and the warps 128 KB at 128 bytes a
// cycle. w B goes through tensor memory for that reason: as a shared-memory operand it cost 160 KB more (149 us
// then, 112 us with it). The rest is latency: a chunk's state chain (ST_GO, decay, S_GO, MMA) and its output
// chain (G_DONE, M, M_GO, M X, Y_DONE, the next G) hand over at barriers, some 110 cycles each, and the warps' work
// between them waits for tensor-memory and shared-memory loads while the roles share the issue slots. D X is added
// by the warps that write the rows, from x loaded ahead of Y (113 us with x loaded beside Y, 117 with D X added as the
// rows are scaled, 123 with one set of warps for both). Measured and not kept, each against 92 to 95 us when D still
// lay on the diagonal: one MMA issuer for all products (112 us); four state warps (102); C as a tensor-memory operand
// (116); polling instead of suspended waits (149); for heads of 128, rows written by the score warps (101).
// Pieces (1 x 131,072 tokens, 32 heads): state pass 351 us, join 16 us, this pass 688 us.
//
// Warp roles (1024 threads; 896 for heads of 64):
//   warp 0       TMA producer (lane 0): x tiles two or three deep, b two, c one or two; tensor memory allocation
//   warp 1       MMA issuer: scores and outputs
//   warp 2       step sizes, running sums and decays of a chunk, one chunk ahead
//   warp 3       MMA issuer: state
//   warps 4-11   scores G -> M (thread = token, two of the four 32-token blocks)
//                then row scaling of C S0^T, half of the columns each
//   warps 12-15  the output rows (thread = token); for heads of 64 the score warps do this too, half of the
//                columns each (16 packed prompts, 32 heads: 286 us against 300)
//   then 8       state: bf16 copy for the next product, decay in place (state channel, half of the columns)
//   last 8       w B, 32 tokens at a time (16 state channels per warp)
// Warp 1 issues C S0^T, M X and the next chunk's C B^T; warp 3 the state product block by block as w B
// comes. Neither waits for the other's order, only for the data (a product of the old state and its decay
// meet in ST_GO and S_GO).
// Tensor memory columns: G (M over it) [0, 128), Y [128, 128 + P), S, then the w B buffers.
#pragma once
#include "kda_ssm_step.cuh"
#include "tcgen05.cuh"

namespace kda {
namespace ssmtc {

using ssm::MIN_LOG2_DECAY;
using ssm::NS;

constexpr int L = 128;          // tokens per chunk
constexpr int SUB = 32;         // tokens per w B block (two MMA steps)
constexpr uint32_t TMEM_COLS = 512;

struct TcParams {
    ssm::SsmParams p;
    int seg_chunks;             // chunks per piece; 0: sequences are not split
    int seg_per_seq;            // pieces per batch row (batched mode)
    int slots;                  // pieces in all
    float *ws;                  // [slots, H, P, NS] states, then [slots, H] log2 decays
};

// per-chunk scalars, two buffers: running log2 sums inside 32-token blocks, the same less log2 delta,
// delta 2^(rest of the block), w, block totals
constexpr int SC_LOC = 0, SC_LD = 512, SC_ES = 1024, SC_W = 1536, SC_TOT = 2048, SC_BYTES = 2112;

template <int P, int PARTS, bool FULL>
struct Layout {
    static constexpr bool MERGED = P == 64;        // the score warps write the output
    static constexpr int EW = MERGED ? 0 : 4, NTHREADS = 32 * (4 + 8 + EW + 8 + 8);
    static constexpr int EC = MERGED ? P / 2 : P;  // columns of an output thread
    static constexpr int WST = 12 + EW, WWB = WST + 8;  // first state and first w B warp
    static constexpr int BOX = L * 128;            // 64 channels x 128 rows, 128-byte swizzle
    static constexpr int XT = P / 64 * BOX, BT = 2 * BOX;
    static constexpr int NSLOT = FULL && PARTS == 3 && P == 128 ? 2 : 4;  // w B buffers of PARTS x 16 columns
    static constexpr int CS = P == 64 ? 2 : 1;     // c tiles in flight
    static constexpr int XS = P == 64 || !FULL ? 3 : 2;  // x tiles in flight (a tile is also its chunk's output buffer)
    static constexpr int BS = FULL ? 2 : 3;        // b tiles in flight
    static constexpr int X = 0;
    static constexpr int B = X + XS * XT;
    static constexpr int C = B + BS * BT;
    static constexpr int H = C + (FULL ? CS * BT : 0);  // bf16 state, [n][p]
    static constexpr int SC = H + (FULL ? XT : 0);
    static constexpr int BAR = SC + 2 * SC_BYTES;
    // YX_GO: the bf16 state is there and Y has been read; M_GO: M is there and Y is scaled; S_GO: the state is
    // decayed; ST_GO: both products of the old state are done; OUT_GO: both products of an x tile are done
    static constexpr int X_FULL = 0, X_EMPTY = 3, OUT_GO = 6, B_FULL = 9, B_EMPTY = 12, C_FULL = 15, C_EMPTY = 17, SC_FULL = 19,
                         SC_EMPTY = 21, G_DONE = 23, M_GO = 24, YX_DONE = 25, Y_DONE = 26, YX_GO = 27, S_GO = 28, ST_GO = 29,
                         X_ZERO = 30, END = 31, END2 = 32, W_FULL = 33, W_EMPTY = 37, NBARS = 42;
    static constexpr int TMEMPTR = BAR + NBARS * 8;
    static constexpr int FLAGS = TMEMPTR + 16;
    static constexpr int ALLOC = FLAGS + 16 + 1024;
    static_assert(ALLOC <= 227 * 1024, "shared memory budget");
    static_assert(SC % 16 == 0 && BAR % 8 == 0 && TMEMPTR % 16 == 0, "alignment");
};

struct Piece {
    int seq, bos, len;      // tokens of the piece
    bool ok, last;          // last piece of its sequence
};

__device__ __forceinline__ int pieces_of(int len, int seg_chunks)
{
    return len <= L * seg_chunks ? 1 : (len + L * seg_chunks - 1) / (L * seg_chunks);
}

// Piece `slot` of a split call: the pieces of the sequences one after another, every lane of a warp
// together (32 sequences per step in varlen mode). Slots past the last piece are not ok.
__device__ __forceinline__ Piece locate(const TcParams &t, int slot)
{
    const ssm::SsmParams &p = t.p;
    int seq, seg;
    if (!p.cu) {
        seq = slot / t.seg_per_seq;
        seg = slot % t.seg_per_seq;
    } else {
        const int lane = threadIdx.x & 31;
        int base = 0;
        seq = -1;
        seg = 0;
        for (int s0 = 0; s0 < p.nseq && seq < 0; s0 += 32) {
            int n = 0;
            if (s0 + lane < p.nseq) {
                const Span sp = ssm::ssm_span(p, s0 + lane);
                n = sp.ok ? pieces_of(sp.len, t.seg_chunks) : 0;
            }
            int inc = n;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, m);
                if (lane >= m) inc += v;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, slot >= base + inc - n && slot < base + inc);
            if (hit) {
                const int src = __ffs(hit) - 1;
                seq = s0 + src;
                seg = slot - base - __shfl_sync(0xffffffffu, inc - n, src);
            }
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (seq < 0) return {0, 0, 0, false, false};
    }
    const Span sp = ssm::ssm_span(p, seq);
    const int span = L * t.seg_chunks;
    const long long at = static_cast<long long>(seg) * span;
    if (at >= sp.len) return {seq, sp.bos, 0, sp.ok && seg == 0, true};  // an empty sequence has one empty piece
    const int len = min(span, sp.len - static_cast<int>(at));
    return {seq, sp.bos + static_cast<int>(at), len, sp.ok, at + len == sp.len};
}

// Varlen order, longest sequences first (up to LPT_MAX_SEQS sequences), so that the long chains start
// in the first wave.
__device__ __forceinline__ int longest_first(const ssm::SsmParams &p, int rank)
{
    const int lane = threadIdx.x & 31;
    int found = rank;
    for (int base = 0; base < p.nseq; base += 32) {
        const int i = base + lane;
        const long long li = i < p.nseq ? p.cu[i + 1] - p.cu[i] : -1;
        int r = 0;
        for (int j = 0; j < p.nseq; ++j) {
            const long long lj = p.cu[j + 1] - p.cu[j];
            r += (lj > li) || (lj == li && j < i);
        }
        const unsigned m = __ballot_sync(0xffffffffu, i < p.nseq && r == rank);
        if (m) found = base + __ffs(m) - 1;
    }
    return found;
}

// The piece of the CTAs of one slot.
__device__ __forceinline__ Piece piece_of(const TcParams &t, int slot)
{
    if (t.seg_chunks) return locate(t, slot);
    const ssm::SsmParams &p = t.p;
    const int seq = p.cu && p.nseq <= LPT_MAX_SEQS ? longest_first(p, slot) : slot;
    const Span sp = ssm::ssm_span(p, seq);
    return {seq, sp.bos, sp.len, sp.ok, true};
}

__device__ __forceinline__ bool no_number(uint32_t fp32_bits) { return (fp32_bits & 0x7f800000u) == 0x7f800000u; }

// What is left of a piece when all its roles are done and some state of it is no number (every thread of the CTA), in
// three steps. Each is out of line: this is rare, and the roles' registers are to stay as they are.
// 1. The first token of every channel whose x is NaN or infinity (`len` where there is none), found row by row.
template <int P, int WARPS>
__device__ __noinline__ void find_spoilt(const ssm::SsmParams &p, int *first, int bos, int len)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint16_t *xp = p.x + static_cast<long long>(bos) * p.xs + static_cast<long long>(blockIdx.x % p.H) * P;
    constexpr int AHEAD = 8;  // loads in flight
    for (int c = threadIdx.x; c < P; c += 32 * WARPS) first[c] = len;
    __syncthreads();
    constexpr int WORDS = P / 64;  // channel pairs per lane
    for (int t0 = warp; t0 < len; t0 += WARPS * AHEAD) {
        uint32_t x[AHEAD][WORDS];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
#pragma unroll
            for (int k = 0; k < WORDS; ++k) {
                const int tok = t0 + WARPS * j;
                x[j][k] = tok < len ? __ldg(reinterpret_cast<const uint32_t *>(xp + tok * p.xs) + 32 * k + lane) : 0u;
            }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
#pragma unroll
            for (int k = 0; k < WORDS; ++k) {
                const int c = 64 * k + 2 * lane;
                if (no_number(x[j][k] << 16)) atomicMin(first + c, t0 + WARPS * j);
                if (no_number(x[j][k])) atomicMin(first + c + 1, t0 + WARPS * j);
            }
    }
}

// 2. The outputs of such a channel from the start of that token's chunk up to the token, made again in fp32: a warp
//    takes channels, four state channels per lane, through the tokens before the chunk and then through the chunk's.
//    Channels whose x holds numbers only are left alone. Inputs are read as constants, so that loads run ahead of stores.
template <int P, int WARPS>
__device__ __noinline__ void repair_spoilt(const TcParams &t, const int *first, int seq, int bos, int len)
{
    const ssm::SsmParams &p = t.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % p.H, slot = blockIdx.x / p.H;
    const size_t unit = static_cast<size_t>(seq) * p.H + h;
    const uint16_t *xp = p.x + static_cast<long long>(bos) * p.xs + static_cast<long long>(h) * P;
    constexpr int AHEAD = 8;  // loads in flight
    constexpr int NC = (P + WARPS - 1) / WARPS;  // channels of a warp
    int start[NC], stop[NC], last = 0;
    float2 s[NC][2];
    auto four = [](const uint16_t *src) { return __ldg(reinterpret_cast<const uint2 *>(src)); };  // of state channels
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = warp + WARPS * k;
        stop[k] = c < P && first[c] < len ? first[c] : 0;
        start[k] = stop[k] / L * L;
        last = max(last, stop[k] > start[k] ? start[k] : 0);
        s[k][0] = s[k][1] = make_float2(0.f, 0.f);
        if (stop[k] == start[k]) continue;
        const size_t row = (unit * P + c) * NS + 4 * lane;
        if (t.seg_chunks || (p.init && p.init_dtype == KDA_DTYPE_FP32)) {
            const float4 v = *reinterpret_cast<const float4 *>(
                t.seg_chunks ? t.ws + ((static_cast<size_t>(slot) * p.H + h) * P + c) * NS + 4 * lane : static_cast<const float *>(p.init) + row);
            s[k][0] = make_float2(v.x, v.y);
            s[k][1] = make_float2(v.z, v.w);
        } else if (p.init) {
            const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.init) + row);
            s[k][0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
            s[k][1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
        }
    }
    const float A2 = -expf(__ldg(p.A_log + h)) * LOG2E, bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f, Dh = p.D ? __ldg(p.D + h) : 0.f;
    const long long grp = static_cast<long long>(h / (p.H / p.G)) * NS + 4 * lane;
    const uint16_t *dp = p.dt + static_cast<long long>(bos) * p.dts + h;
    const uint16_t *bp = p.b + static_cast<long long>(bos) * p.bs + grp, *cp = p.c + static_cast<long long>(bos) * p.cs + grp;
    uint16_t *op = p.out + static_cast<long long>(bos) * p.os + static_cast<long long>(h) * P;
    uint32_t xn[NC], dn = 0u;  // of the lane's token of 32, fetched ahead
    auto fetch = [&](int tok) {
        dn = __ldg(dp + tok * p.dts);
#pragma unroll
        for (int k = 0; k < NC; ++k) xn[k] = warp + WARPS * k < P ? __ldg(xp + tok * p.xs + warp + WARPS * k) : 0u;
    };
    auto step = [](float2(&v)[2], float keep, float dx, const uint2 &b) {
        v[0] = ffma2(make_float2(keep, keep), v[0], fmul2(make_float2(dx, dx), make_float2(bf16_lo(b.x), bf16_hi(b.x))));
        v[1] = ffma2(make_float2(keep, keep), v[1], fmul2(make_float2(dx, dx), make_float2(bf16_lo(b.y), bf16_hi(b.y))));
    };
    if (last > 0) fetch(lane);
    for (int t0 = 0; t0 < last; t0 += 32) {
        const float delta = ssm::softplus(__uint_as_float(dn << 16) + bias), keep = exp2f(A2 * delta);
        float dx[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) dx[k] = delta * __uint_as_float(xn[k] << 16);
        fetch(min(t0 + 32, last - 32) + lane);
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += AHEAD) {
            uint2 b[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) b[i] = four(bp + (t0 + i0 + i) * p.bs);
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                if (t0 >= start[k]) continue;
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) step(s[k], __shfl_sync(0xffffffffu, keep, i0 + i), __shfl_sync(0xffffffffu, dx[k], i0 + i), b[i]);
            }
        }
    }
#pragma unroll 1
    for (int k = 0; k < NC; ++k) {
        const int c = warp + WARPS * k;
        float2 v[2] = {s[0][0], s[0][1]};
        int from = start[0], to = stop[0];
#pragma unroll
        for (int j = 1; j < NC; ++j)
            if (j == k) {
                v[0] = s[j][0];
                v[1] = s[j][1];
                from = start[j];
                to = stop[j];
            }
        for (int t0 = from; t0 < to; t0 += 32) {
            const int n = min(32, to - t0), own = t0 + min(lane, n - 1);
            const float x = __uint_as_float(static_cast<uint32_t>(__ldg(xp + own * p.xs + c)) << 16);
            const float delta = ssm::softplus(__uint_as_float(static_cast<uint32_t>(__ldg(dp + own * p.dts)) << 16) + bias);
            const float keep = exp2f(A2 * delta), dx = delta * x;
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const uint2 b = four(bp + (t0 + i) * p.bs), q = four(cp + (t0 + i) * p.cs);
                step(v, __shfl_sync(0xffffffffu, keep, i), __shfl_sync(0xffffffffu, dx, i), b);
                const float2 u = ffma2(v[0], make_float2(bf16_lo(q.x), bf16_hi(q.x)), fmul2(v[1], make_float2(bf16_lo(q.y), bf16_hi(q.y))));
                float y = u.x + u.y;
#pragma unroll
                for (int m = 16; m >= 1; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
                if (lane == i) op[(t0 + i) * p.os + c] = f2bf_bits(p.D ? fmaf(Dh, x, y) : y);
            }
        }
    }
}

// Whether some lane of the warp holds a value that is no number (0 NaN and 0 inf are NaN).
__device__ __forceinline__ bool any_spoilt(const uint32_t (&r)[32])
{
    float2 z = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 32; i += 2) z = ffma2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), make_float2(0.f, 0.f), z);
    return __any_sync(0xffffffffu, !(z.x + z.y == 0.f));
}

// 3. Final states of which a warp holds some that are no numbers: until here they have left the initial state, maybe the
//    same buffer, to step 2. 32 columns of the state in tensor memory at `taddr`, to the final state's elements from
//    `first` on.
__device__ __noinline__ void store_spoilt(const ssm::SsmParams &p, uint32_t taddr, size_t first)
{
    const size_t st_elems = static_cast<size_t>(p.nseq) * p.H * p.P * NS;
    uint32_t r[32];
    tc::ld32(taddr, r);
    tc::wait_ld();
    if (!any_spoilt(r)) return;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const size_t at = first + static_cast<size_t>(i) * NS;
        if (!gmem_ok(at, 1, st_elems)) continue;
        if (p.fin_dtype == KDA_DTYPE_FP32)
            static_cast<float *>(p.fin)[at] = __uint_as_float(r[i]);
        else
            static_cast<uint16_t *>(p.fin)[at] = f2bf_bits(__uint_as_float(r[i]));
    }
}

template <int P, int PARTS>
__device__ __noinline__ void finish_spoilt(const TcParams &t)
{
    using Lay = Layout<P, PARTS, true>;
    constexpr int WARPS = Lay::NTHREADS / 32;
    __shared__ int first[P];
    const Piece pc = piece_of(t, blockIdx.x / t.p.H);
    find_spoilt<P, WARPS>(t.p, first, pc.bos, pc.len);
    __syncthreads();
    repair_spoilt<P, WARPS>(t, first, pc.seq, pc.bos, pc.len);
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (pc.last && t.p.fin && warp >= Lay::WST && warp < Lay::WST + 8) {  // the state warps
        const int q = warp & 3, c0 = warp < Lay::WST + 4 ? 0 : P / 2;
        __syncwarp();
        tc::fence_after();
        for (int c = c0; c < c0 + P / 2; c += 32)
            store_spoilt(t.p, (static_cast<uint32_t>(32 * q) << 16) + 128 + P + c,
                       ((static_cast<size_t>(pc.seq) * t.p.H + blockIdx.x % t.p.H) * P + c) * NS + 32 * q + lane);
        tc::fence_before();
    }
    __syncthreads();
}

// FULL: outputs and states; else only the state that the piece leaves when it starts from zero (to
// the workspace, with its decay), for the pieces that another one follows. That state is one sum over the
// piece's tokens, each weighted by the decay from it to the piece's end, so the chunks are taken from the
// last to the first: the weights follow from a running sum, and the accumulator is never decayed, so no
// chunk waits for the one before it.
template <int P, int PARTS, bool FULL>
__global__ void __launch_bounds__(Layout<P, PARTS, FULL>::NTHREADS, 1)
    kda_ssm_tc_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tb,
                      const __grid_constant__ CUtensorMap tcm, const __grid_constant__ CUtensorMap to, const __grid_constant__ TcParams t)
{
    using Lay = Layout<P, PARTS, FULL>;
    constexpr int CS = Lay::CS, XS = Lay::XS, BS = Lay::BS, OUTW = Lay::MERGED ? 8 : 4;  // OUTW: warps that write the output
    constexpr uint32_t T_G = 0, T_Y = FULL ? 128 : 0, T_S = T_Y + (FULL ? P : 0), T_W = T_S + P;
    static_assert(T_W + Lay::NSLOT * PARTS * (SUB / 2) <= TMEM_COLS, "tensor memory budget");
    extern __shared__ uint8_t smem_dyn[];
    uint8_t *smem = smem_dyn + ((1024u - (smem_u32(smem_dyn) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
#define SM_AT(T, a) (*reinterpret_cast<T *>(smem + (smem_checked((a), sizeof(T), sb) - sb)))
    const ssm::SsmParams &p = t.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % p.H, slot = blockIdx.x / p.H;
    const Piece pc = piece_of(t, slot);
    if (FULL && p.cu && blockIdx.x == 0) blk::check_bounds(p.cu, p.nseq, p.total);
    if (!pc.ok || (!FULL && pc.last)) return;  // CTA-uniform, before any tensor memory is taken
    const int nch = (pc.len + L - 1) / L;
    const int grp = h / (p.H / p.G);

    volatile int *flags = reinterpret_cast<volatile int *>(smem + Lay::FLAGS);
    __shared__ volatile uint32_t spoilt;  // some state at the end of the piece is no number
    auto bar = [&](int i) { return sb + Lay::BAR + 8 * i; };
    auto xt = [&](int n) { return sb + Lay::X + (n % XS) * Lay::XT; };
    auto bt = [&](int n) { return sb + Lay::B + (n % BS) * Lay::BT; };
    auto ct = [&](int n) { return sb + Lay::C + (n % CS) * Lay::BT; };
    auto sc = [&](int n) { return sb + Lay::SC + (n & 1) * SC_BYTES; };
    // step n is chunk n, or the n-th from the end
    auto chunk_of = [&](int n) { return FULL ? n : nch - 1 - n; };
    auto live_of = [&](int n) { return min(L, pc.len - chunk_of(n) * L); };

    if (warp == 0) {
        tc::alloc(sb + Lay::TMEMPTR, TMEM_COLS);
        tc::relinquish();
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < XS; ++i) {
            mbar_init(bar(Lay::X_FULL + i), 1);
            mbar_init(bar(Lay::X_EMPTY + i), FULL ? OUTW : 1);
            mbar_init(bar(Lay::OUT_GO + i), 2);
        }
        for (int i = 0; i < BS; ++i) {
            mbar_init(bar(Lay::B_FULL + i), 1);
            mbar_init(bar(Lay::B_EMPTY + i), FULL ? 9 : 16);  // the w B warps, and the score product
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(Lay::C_FULL + i), 1);
            mbar_init(bar(Lay::C_EMPTY + i), 1);
            mbar_init(bar(Lay::SC_FULL + i), 1);
            mbar_init(bar(Lay::SC_EMPTY + i), FULL ? 24 : 16);
        }
        for (int i : {Lay::G_DONE, Lay::YX_DONE, Lay::Y_DONE, Lay::END, Lay::END2}) mbar_init(bar(i), 1);
        for (int i : {Lay::S_GO, Lay::X_ZERO}) mbar_init(bar(i), 8);
        mbar_init(bar(Lay::M_GO), 8);
        mbar_init(bar(Lay::YX_GO), 8 + OUTW);
        mbar_init(bar(Lay::ST_GO), FULL ? 2 : 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(Lay::W_FULL + i), 8);
            mbar_init(bar(Lay::W_EMPTY + i), 1);
        }
        flags[0] = 0;
        spoilt = 0u;
        fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    // The allocation is the whole tensor memory, so it starts at address 0: as a constant, it leaves the
    // MMA operands constants too.
    constexpr uint32_t tmem = 0;
    if (*reinterpret_cast<volatile uint32_t *>(smem + Lay::TMEMPTR) != tmem && threadIdx.x == 0) {
        atomicOr(&g_dev_error, DEVERR_TIMEOUT);
        flags[0] = 1;
    }
    // the whole warp goes on only when every lane saw the phase (a wait on a phase that is over already costs
    // about 100 cycles, so the roles' critical waits are few)
    auto wait_w = [&](int b, uint32_t par) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar(b), par))) return true;
        const bool ok = __all_sync(0xffffffffu, wait_bar_slow(bar(b), par, flags));
        __syncwarp();
        return ok;
    };
    auto arrive_w = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b));
    };

    // The output's two steps, for a thread's token (quarter q, lane).
    // Y = C S0^T times the decay from the chunk's start to the token, in place, half of the columns:
    auto scale_rows = [&](uint32_t ly, float e) {
#pragma unroll 1
        for (int g4 = 0; g4 < P / 64; ++g4) {
            uint32_t y[32];
            tc::ld32(ly + 32 * g4, y);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 v = fmul2(make_float2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), make_float2(e, e));
                y[i] = __float_as_uint(v.x);
                y[i + 1] = __float_as_uint(v.y);
            }
            tc::st32(ly + 32 * g4, y);
        }
        tc::wait_st();
        tc::fence_before();
        arrive_w(Lay::M_GO);
    };
    // Y + D x, summed in fp32, to bf16, over the x tile (both products have read it, and a thread reads its own elements
    // of it first) and from there to memory by TMA, 32 tokens per warp; a ragged end is stored from registers.
    const float Dh = p.D ? __ldg(p.D + h) : 0.f;
    auto row_at = [&](int n, int row, int c) { return xt(n) + (c >> 6) * Lay::BOX + row * 128; };
    auto group_at = [&](int row, int c, int i) { return ((((c >> 3) & 7) + i) ^ (row & 7)) << 4; };  // eight channels, swizzled by the row
    auto load_x = [&](int n, int q, int c, uint4(&x)[4]) {  // channels c .. c + 31
        const int row = 32 * q + lane;
        const uint32_t xr = row_at(n, row, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = SM_AT(const uint4, xr + group_at(row, c, i));
    };
    // x holds the first 32 columns' elements already; the next ones' are loaded while these are stored.
    auto write_rows = [&](uint32_t ly, int n, int q, int c0, uint4(&x)[4]) {
        const int row = 32 * q + lane, Lv = live_of(n);
        uint16_t *op = p.out + static_cast<long long>(pc.bos + n * L + row) * p.os + static_cast<long long>(h) * P;
#pragma unroll 1
        for (int g4 = 0; g4 < Lay::EC / 32; ++g4) {
            const int c = c0 + 32 * g4;
            const uint32_t xr = row_at(n, row, c);
            uint32_t y[32], o[16];
            tc::ld32(ly + 32 * g4, y);
            tc::wait_ld();
            if (g4 + 1 == Lay::EC / 32) {
                tc::fence_before();
                arrive_w(Lay::YX_GO);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 f[4];
                blk::unpack8(x[i], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = ffma2(make_float2(Dh, Dh), f[j], make_float2(__uint_as_float(y[8 * i + 2 * j]), __uint_as_float(y[8 * i + 2 * j + 1])));
                    o[4 * i + j] = pack_bf16(v.x, v.y);
                }
            }
            if (g4 + 1 < Lay::EC / 32) load_x(n, q, c + 32, x);
            if (Lv == L) {
#pragma unroll
                for (int i = 0; i < 4; ++i) SM_AT(uint4, xr + group_at(row, c, i)) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            } else if (row < Lv) {
#pragma unroll
                for (int i = 0; i < 4; ++i) reinterpret_cast<uint4 *>(op + c)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
        }
        if (Lv == L) {
            tc::fence_async_smem();
            if constexpr (Lay::MERGED) named_bar_sync(1 + q, 64);  // two warps fill the rows; the first stores them
            __syncwarp();
            if (lane == 0 && c0 == 0) {
#pragma unroll
                for (int k = 0; k < P / 64; ++k)
                    tma_store_3d(&to, xt(n) + k * Lay::BOX + 32 * q * 128, 64 * k, h, pc.bos + n * L + 32 * q);
                bulk_commit();
            }
        }
    };
    // ... and once the store has read the tile it is free for another chunk's x
    auto release_rows = [&](int n) {
        if (lane == 0) bulk_wait_read();
        arrive_w(Lay::X_EMPTY + n % XS);
    };

    // w B: warp wi of eight, every GROUPS-th block from `group` on (a piece that only leaves its state has whole
    // chunks alone, so only one group ever meets a ragged one)
    constexpr int GROUPS = FULL ? 1 : 2;
    auto make_wb = [&](int wi, int group) {
        // A warp owns 16 state channels. ldmatrix.trans hands a lane two tokens of one
        // channel, the layout in which the 16-lane tensor-memory stores take them, so the transposition is free.
        const int u = 32 * wi + lane, ch16 = 2 * (warp & 3) + (wi < 4 ? 0 : 1);
        const uint32_t lb = tmem + (static_cast<uint32_t>(16 * ch16) << 16) + T_W;
        const int c8 = 2 * ch16 + ((lane >> 3) & 1);  // eight-channel group of this lane's address
        // matrix lane >> 3 of an ldmatrix: tokens 8 (lane >> 4) .., channels 8 ((lane >> 3) & 1) ..
        const int jr = 8 * (lane >> 4) + (lane & 7);
        int k = 0;
        bool ok = true;
        for (int n = 0; ok && n < nch; ++n) {
            const int Lv = live_of(n), nsub = (Lv + SUB - 1) / SUB;
            ok = wait_w(Lay::SC_FULL + (n & 1), (n >> 1) & 1) && wait_w(Lay::B_FULL + n % BS, (n / BS) & 1);
            if (ok && Lv < L) {
                // rows past the end hold another sequence's tokens: zero, so that a NaN there meets no product
                ok = wait_w(Lay::X_FULL + n % XS, (n / XS) & 1);
                if (ok)
                    for (int i = u; i < (L - Lv) * (P / 8); i += 256) {
                        const int r = Lv + i / (P / 8), c8 = i % (P / 8);
                        SM_AT(uint4, xt(n) + (c8 >> 3) * Lay::BOX + r * 128 + (c8 & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                tc::fence_async_smem();
                if (ok) arrive_w(Lay::X_ZERO);
            }
            for (int s = group; ok && s < nsub; s += GROUPS) {
                const int sl = (k + s) % Lay::NSLOT, j0 = SUB * s;
                float2 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = SM_AT(const float2, sc(n) + SC_W + 4 * (j0 + 8 * i + 2 * (lane & 3)));
                uint32_t v[8];
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // tokens j0 + 16 i ..
                    const int j = j0 + 16 * i + jr;
                    ldsm_x4_t(bt(n) + (c8 >> 3) * Lay::BOX + j * 128 + (((c8 & 7) ^ (j & 7)) << 4), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
                if (Lv < L) {  // past the end b may be anything
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = j0 + 8 * (i >> 1) + 2 * (lane & 3);
                        v[i] &= j + 1 < Lv ? 0xffffffffu : j < Lv ? 0xffffu : 0u;
                    }
                }
                float2 f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = fmul2(make_float2(bf16_lo(v[i]), bf16_hi(v[i])), w[i >> 1]);
                // everything is at hand in registers before the buffer is waited for
                uint32_t o[PARTS][8];
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (part + 1 < PARTS) {  // the upper eight bits; what is left is exact
                            const uint32_t a = __float_as_uint(f[i].x), b = __float_as_uint(f[i].y);
                            o[part][i] = __byte_perm(a, b, 0x7632);
                            f[i] = fsub2(f[i], make_float2(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u)));
                        } else {
                            o[part][i] = pack_bf16(f[i].x, f[i].y);
                        }
                    }
                ok = wait_w(Lay::W_EMPTY + sl, (((k + s) / Lay::NSLOT) & 1) ^ 1);
                if (!ok) break;
                tc::fence_after();
#pragma unroll
                for (int part = 0; part < PARTS; ++part) tc::st_16x128b_x4(lb + (sl * PARTS + part) * (SUB / 2), o[part]);
                tc::wait_st();
                tc::fence_before();
                arrive_w(Lay::W_FULL + sl);
            }
            k += nsub;
            if (ok) {
                arrive_w(Lay::B_EMPTY + n % BS);
                arrive_w(Lay::SC_EMPTY + (n & 1));
            }
        }
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        if (lane == 0) {
            tma_prefetch_desc(&tx);
            tma_prefetch_desc(&tb);
            if (FULL) tma_prefetch_desc(&tcm);
            int nb = 0, nx = 0, ncc = 0;  // tiles issued
            for (int n = 0; n < nch; ++n) {
                const int s = n % BS, tok = pc.bos + chunk_of(n) * L;
                if (!wait_bar(bar(Lay::B_EMPTY + s), ((n / BS) & 1) ^ 1, flags)) break;
                mbar_arrive_expect_tx(bar(Lay::B_FULL + s), Lay::BT);
#pragma unroll
                for (int k = 0; k < 2; ++k) tma_load_3d(bt(n) + k * Lay::BOX, &tb, 64 * k, grp, tok, bar(Lay::B_FULL + s));
                ++nb;
                if constexpr (FULL) {
                    if (!wait_bar(bar(Lay::C_EMPTY + n % CS), ((n / CS) & 1) ^ 1, flags)) break;
                    mbar_arrive_expect_tx(bar(Lay::C_FULL + n % CS), Lay::BT);
#pragma unroll
                    for (int k = 0; k < 2; ++k) tma_load_3d(ct(n) + k * Lay::BOX, &tcm, 64 * k, grp, tok, bar(Lay::C_FULL + n % CS));
                    ++ncc;
                }
                const int xs = n % XS;
                if (!wait_bar(bar(Lay::X_EMPTY + xs), ((n / XS) & 1) ^ 1, flags)) break;
                mbar_arrive_expect_tx(bar(Lay::X_FULL + xs), Lay::XT);
#pragma unroll
                for (int k = 0; k < P / 64; ++k) tma_load_3d(xt(n) + k * Lay::BOX, &tx, 64 * k, h, tok, bar(Lay::X_FULL + xs));
                ++nx;
            }
            // no copy is in flight when the CTA ends, whichever way the loop was left
            for (int m = nb > BS ? nb - BS : 0; m < nb; ++m) drain_bar(bar(Lay::B_FULL + m % BS), (m / BS) & 1);
            for (int m = nx > XS ? nx - XS : 0; m < nx; ++m) drain_bar(bar(Lay::X_FULL + m % XS), (m / XS) & 1);
            for (int m = ncc > CS ? ncc - CS : 0; m < ncc; ++m) drain_bar(bar(Lay::C_FULL + m % CS), (m / CS) & 1);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer: scores and outputs (whole warp)
        if (FULL && nch > 0) {
            constexpr uint32_t id_g = tc::idesc(tc::BF16, 128, 128, 0, 0);
            constexpr uint32_t id_y = tc::idesc(tc::BF16, 128, P, 0, 1);
            constexpr uint32_t HI = tc::sdesc_hi(1024, tc::SWZ_128B);
            const uint32_t dh = tc::sdesc_lo(sb + Lay::H, Lay::BOX);
            auto kmaj = [&](uint32_t lo, int i) {  // K step i of a K-major tile (two boxes of 64 channels)
                return tc::sdesc_of<HI>(lo + static_cast<uint32_t>(((i >> 2) * Lay::BOX + (i & 3) * 32) >> 4));
            };
            auto nmaj = [&](uint32_t lo, int i) {  // K step i (16 rows) of an MN-major tile
                return tc::sdesc_of<HI>(lo + static_cast<uint32_t>(i * ((16 * 128) >> 4)));
            };
            auto issue_g = [&](int n) {  // its tensor memory holds the M of the last chunk until that has been read
                if (!wait_w(Lay::B_FULL + n % BS, (n / BS) & 1) || !wait_w(Lay::C_FULL + n % CS, (n / CS) & 1)) return false;
                if (n > 0 && !wait_w(Lay::Y_DONE, (n - 1) & 1)) return false;
                tc::fence_after();
                const uint32_t dc = tc::sdesc_lo(ct(n), 16), db = tc::sdesc_lo(bt(n), 16);
#pragma unroll
                for (int i = 0; i < 8; ++i) tc::mma_ss_w(tmem + T_G, kmaj(dc, i), kmaj(db, i), id_g, i > 0);
                tc::commit_w(bar(Lay::G_DONE));
                tc::commit_w(bar(Lay::B_EMPTY + n % BS));
                return true;
            };
            bool ok = issue_g(0);
            for (int n = 0; ok && n < nch; ++n) {
                const uint32_t dx = tc::sdesc_lo(xt(n), Lay::BOX), dc = tc::sdesc_lo(ct(n), 16);
                // Y = C S0^T, over the accumulator whose last values have been read
                ok = wait_w(Lay::X_FULL + n % XS, (n / XS) & 1) && wait_w(Lay::YX_GO, n & 1);
                if (!ok) break;
                tc::fence_after();
#pragma unroll
                for (int i = 0; i < 8; ++i) tc::mma_ss_w(tmem + T_Y, kmaj(dc, i), nmaj(dh, i), id_y, i > 0);
                tc::commit_w(bar(Lay::YX_DONE));
                tc::commit_w(bar(Lay::ST_GO));
                tc::commit_w(bar(Lay::C_EMPTY + n % CS));
                // Y += M X
                ok = (live_of(n) == L || wait_w(Lay::X_ZERO, 0)) && wait_w(Lay::M_GO, n & 1);
                if (!ok) break;
                tc::fence_after();
#pragma unroll
                for (int i = 0; i < 8; ++i) tc::mma_ts_w(tmem + T_Y, tmem + T_G + 64 * (i >> 2) + 8 * (i & 3), nmaj(dx, i), id_y, 1);
                tc::commit_w(bar(Lay::OUT_GO + n % XS));
                tc::commit_w(bar(Lay::Y_DONE));
                if (n + 1 < nch) ok = issue_g(n + 1);
            }
            tc::commit_w(bar(Lay::END));
            if (lane == 0) drain_bar(bar(Lay::END), 0);
            __syncwarp();
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------- step sizes and decays
        const float A2 = -expf(__ldg(p.A_log + h)) * LOG2E, bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f;
        const uint16_t *dp = p.dt + static_cast<long long>(pc.bos) * p.dts + h;
        const int j0 = 4 * lane;
        uint32_t raw[4] = {0u, 0u, 0u, 0u};
        auto fetch = [&](int n) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n < nch && chunk_of(n) * L + j0 + i < pc.len) raw[i] = dp[static_cast<long long>(chunk_of(n) * L + j0 + i) * p.dts];
        };
        fetch(0);
        float seg = 0.f;
        for (int n = 0; n < nch; ++n) {
            const int Lv = live_of(n);
            float d[4], a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool live = j0 + i < Lv;
                d[i] = live ? ssm::softplus(__uint_as_float(raw[i] << 16) + bias) : 0.f;
                const float u = A2 * d[i];  // held at the least decay by a comparison that lets NaN through (fmaxf would not)
                a[i] = !live ? 0.f : u < MIN_LOG2_DECAY ? MIN_LOG2_DECAY : u;
            }
            fetch(n + 1);
            // running sums inside the lane, then over the eight lanes of a block, from both ends
            const float l0 = a[0], l1 = l0 + a[1], l2 = l1 + a[2], l3 = l2 + a[3];
            const float r3 = 0.f, r2 = a[3], r1 = a[2] + r2, r0 = a[1] + r1;
            float pre = l3, post = l3;
#pragma unroll
            for (int m = 1; m < 8; m <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, pre, m, 8), v = __shfl_down_sync(0xffffffffu, post, m, 8);
                if ((lane & 7) >= m) pre += u;
                if ((lane & 7) + m < 8) post += v;
            }
            float before = __shfl_up_sync(0xffffffffu, pre, 1, 8), after = __shfl_down_sync(0xffffffffu, post, 1, 8);
            if ((lane & 7) == 0) before = 0.f;
            if ((lane & 7) == 7) after = 0.f;
            const float t0 = __shfl_sync(0xffffffffu, pre, 7), t1 = __shfl_sync(0xffffffffu, pre, 15);
            const float t2 = __shfl_sync(0xffffffffu, pre, 23), t3 = __shfl_sync(0xffffffffu, pre, 31);
            const int blkq = lane >> 3;
            const float rest = (blkq == 0 ? t1 + (t2 + t3) : blkq == 1 ? t2 + t3 : blkq == 2 ? t3 : 0.f) + (FULL ? 0.f : seg);
            seg += (t0 + t1) + (t2 + t3);
            const float sf[4] = {r0 + after, r1 + after, r2 + after, r3 + after};
            if (!wait_w(Lay::SC_EMPTY + (n & 1), ((n >> 1) & 1) ^ 1)) break;
            const uint32_t o = sc(n) + 4 * j0;
            SM_AT(float4, o + SC_LOC) = make_float4(before + l0, before + l1, before + l2, before + l3);
            // running sum less log2 delta (delta 0: no score at all)
            SM_AT(float4, o + SC_LD) = make_float4(before + l0 - lg2_approx(d[0]), before + l1 - lg2_approx(d[1]), before + l2 - lg2_approx(d[2]), before + l3 - lg2_approx(d[3]));
            SM_AT(float4, o + SC_ES) = make_float4(d[0] * ex2_approx(sf[0]), d[1] * ex2_approx(sf[1]), d[2] * ex2_approx(sf[2]), d[3] * ex2_approx(sf[3]));
            SM_AT(float4, o + SC_W) = make_float4(d[0] * ex2_approx(sf[0] + rest), d[1] * ex2_approx(sf[1] + rest),
                                                  d[2] * ex2_approx(sf[2] + rest), d[3] * ex2_approx(sf[3] + rest));
            if (lane == 0) SM_AT(float4, sc(n) + SC_TOT) = make_float4(t0, t1, t2, t3);
            arrive_w(Lay::SC_FULL + (n & 1));
        }
        if (!FULL && lane == 0)
            t.ws[static_cast<size_t>(t.slots) * p.H * P * NS + static_cast<size_t>(slot) * p.H + h] = seg;
    } else if (warp == 3) {
        // ---------------------------------------------------------------- MMA issuer: state
        if (nch > 0) {
            constexpr uint32_t id_s = tc::idesc(tc::BF16, 128, P, 0, 1), HI = tc::sdesc_hi(1024, tc::SWZ_128B);
            int k = 0;  // w B blocks so far
            bool ok = true;
            for (int n = 0; ok && n < nch; ++n) {
                const int nsub = (live_of(n) + SUB - 1) / SUB;
                uint32_t dx = tc::sdesc_lo(xt(n), Lay::BOX);
                // (the first block's wait comes before the one that is on the chain)
                ok = wait_w(Lay::X_FULL + n % XS, (n / XS) & 1) && wait_w(Lay::W_FULL + k % Lay::NSLOT, (k / Lay::NSLOT) & 1) &&
                     (!FULL && n > 0 ? true : wait_w(Lay::S_GO, n & 1));
                for (int s = 0; ok && s < nsub; ++s, ++k, dx += (SUB * 128) >> 4) {
                    const int sl = k % Lay::NSLOT;
                    ok = s == 0 || wait_w(Lay::W_FULL + sl, (k / Lay::NSLOT) & 1);
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t wb = tmem + T_W + sl * (PARTS * (SUB / 2));
#pragma unroll
                    for (int i = 0; i < PARTS; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            tc::mma_ts_w(tmem + T_S, wb + i * (SUB / 2) + 8 * j, tc::sdesc_of<HI>(dx + ((j * 16 * 128) >> 4)), id_s, 1);
                    tc::commit_w(bar(Lay::W_EMPTY + sl));
                }
                if (!ok) break;
                if (FULL || n + 1 == nch) tc::commit_w(bar(Lay::ST_GO));
                tc::commit_w(bar((FULL ? Lay::OUT_GO : Lay::X_EMPTY) + n % XS));
            }
            tc::commit_w(bar(Lay::END2));
            if (lane == 0) drain_bar(bar(Lay::END2), 0);
            __syncwarp();
            // NaN or infinity in x leaves no number in its whole column of the state, and for good (0 NaN and 0 inf are
            // NaN): this warp's lanes show it.
            if (FULL && ok) {
                tc::fence_after();
#pragma unroll 1
                for (int g4 = 0; g4 < P / 32; ++g4) {
                    uint32_t r[32];
                    tc::ld32(tmem + (static_cast<uint32_t>(32 * 3) << 16) + T_S + 32 * g4, r);
                    tc::wait_ld();
                    if (any_spoilt(r)) spoilt = 1u;
                }
                tc::fence_before();
            }
        }
    } else if (warp < 12) {
        // ---------------------------------------------------------------- scores
        if constexpr (FULL) {
            // This thread's columns are blocks 2 hf and 2 hf + 1 of its token's row; M is written over columns
            // of G that it has read itself (the product takes M's halves from columns 0 and 64).
            const int q = warp & 3, row = 32 * q + lane, hf = warp < 8 ? 0 : 1;
            const uint32_t lb = tmem + (static_cast<uint32_t>(32 * q) << 16) + T_G + 64 * hf;
            const int c0 = hf * (P / 2);  // Y columns that this warp scales and, for heads of 64, writes
            const uint32_t ly = tmem + (static_cast<uint32_t>(32 * q) << 16) + T_Y + c0;
            if (Lay::MERGED) arrive_w(Lay::YX_GO);  // nothing of Y is waiting to be read
            const int nfull = min(max(2 * (q - 2 * hf), 0), 4), nlive = min(max(2 * (q - 2 * hf) + 2, 0), 4);
            for (int n = 0; n < nch; ++n) {
                if (!wait_w(Lay::SC_FULL + (n & 1), (n >> 1) & 1)) break;
                const float4 tot = SM_AT(const float4, sc(n) + SC_TOT);
                const float loc = SM_AT(const float, sc(n) + SC_LOC + 4 * row);
                // log2 decay from the end of the second and of the first block to this row
                const float l1 = loc + (q == 3 && hf == 0 ? tot.z : 0.f);
                const float e1 = ex2_approx(l1), e0 = ex2_approx(l1 + (q >= 2 && hf == 0 ? tot.y : 0.f));
                uint32_t s = sc(n) + 256 * hf;
                if constexpr (Lay::MERGED) {  // x is read as the rows are written: waited for here, ahead of the chain
                    if (!wait_w(Lay::X_FULL + n % XS, (n / XS) & 1)) break;
                    if (n > 0) release_rows(n - 1);
                }
                if (!wait_w(Lay::G_DONE, n & 1)) break;
                tc::fence_after();
#pragma unroll 1
                for (int b = 0; b < nfull; ++b) {
                    uint32_t g[16], m[8];
                    tc::ld16(lb + 16 * b, g);
                    const float2 e = b < 2 ? make_float2(e0, e0) : make_float2(e1, e1);
                    float2 u[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = SM_AT(const float4, s + SC_ES + 64 * b + 16 * i);
                        u[2 * i] = fmul2(make_float2(v.x, v.y), e);
                        u[2 * i + 1] = fmul2(make_float2(v.z, v.w), e);
                    }
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 o = fmul2(u[i], make_float2(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1])));
                        m[i] = pack_bf16(o.x, o.y);
                    }
                    tc::st8(lb + 8 * b, m);
                }
#pragma unroll 1
                for (int b = nfull; b < nlive; ++b) {
                    uint32_t g[16], m[8];
                    tc::ld16(lb + 16 * b, g);
                    const int col = lane - 16 * (b & 1);  // this row's own column in the piece
                    float w[16];
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 v = SM_AT(const float4, s + SC_LD + 64 * b + 4 * i);
                        w[i] = ex2_approx(loc - v.x);
                        w[i + 1] = ex2_approx(loc - v.y);
                        w[i + 2] = ex2_approx(loc - v.z);
                        w[i + 3] = ex2_approx(loc - v.w);
                    }
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = i <= col ? w[i] * __uint_as_float(g[i]) : 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) m[i] = pack_bf16(w[2 * i], w[2 * i + 1]);
                    tc::st8(lb + 8 * b, m);
                }
                if (nlive < 4) {
                    const uint32_t z[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll 1
                    for (int b = nlive; b < 4; ++b) tc::st8(lb + 8 * b, z);
                }
                tc::wait_st();
                const float e = ex2_approx(loc + (q > 0 ? tot.x : 0.f) + (q > 1 ? tot.y : 0.f) + (q > 2 ? tot.z : 0.f));
                arrive_w(Lay::SC_EMPTY + (n & 1));
                if (!wait_w(Lay::YX_DONE, n & 1)) break;
                tc::fence_after();
                scale_rows(ly, e);
                if constexpr (Lay::MERGED) {
                    uint4 x[4];
                    load_x(n, q, c0, x);
                    if (!wait_w(Lay::OUT_GO + n % XS, (n / XS) & 1)) break;
                    tc::fence_after();
                    write_rows(ly, n, q, c0, x);
                }
            }
            if (Lay::MERGED && lane == 0) bulk_wait_all();
        } else {
            make_wb(warp - 4, 0);  // no scores here: these warps share the work on w B
        }
    } else if (warp < Lay::WST) {
        // ---------------------------------------------------------------- outputs
        if constexpr (FULL && !Lay::MERGED) {
            const int q = warp & 3;
            const uint32_t ly = tmem + (static_cast<uint32_t>(32 * q) << 16) + T_Y;
            arrive_w(Lay::YX_GO);  // nothing of Y is waiting to be read
            for (int n = 0; n < nch; ++n) {
                if (!wait_w(Lay::X_FULL + n % XS, (n / XS) & 1)) break;
                uint4 x[4];
                load_x(n, q, 0, x);
                if (!wait_w(Lay::OUT_GO + n % XS, (n / XS) & 1)) break;
                tc::fence_after();
                write_rows(ly, n, q, 0, x);
                release_rows(n);
            }
            if (lane == 0) bulk_wait_all();
        }
    } else if (warp < Lay::WWB) {
        // ---------------------------------------------------------------- state
        const int q = warp & 3, nn = 32 * q + lane, c0 = warp < Lay::WST + 4 ? 0 : P / 2;  // this thread's channel and columns
        const uint32_t lb = tmem + (static_cast<uint32_t>(32 * q) << 16) + T_S + c0;
        const size_t unit = static_cast<size_t>(pc.seq) * p.H + h;
        const size_t st_elems = static_cast<size_t>(p.nseq) * p.H * P * NS;
        float *wsp = t.seg_chunks ? t.ws + (static_cast<size_t>(slot) * p.H + h) * P * NS + nn : nullptr;
        // 32 columns (head channels c0 + 32 g4 ..) of the state this piece starts from
        auto load_init = [&](int g4, uint32_t(&r)[32]) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const size_t at = static_cast<size_t>(c0 + 32 * g4 + i) * NS;
                r[i] = 0u;
                if constexpr (!FULL) continue;
                if (t.seg_chunks) {
                    r[i] = __float_as_uint(wsp[at]);
                } else if (p.init && gmem_ok(unit * P * NS + at + nn, 1, st_elems)) {
                    r[i] = p.init_dtype == KDA_DTYPE_FP32
                               ? __float_as_uint(static_cast<const float *>(p.init)[unit * P * NS + at + nn])
                               : static_cast<uint32_t>(static_cast<const uint16_t *>(p.init)[unit * P * NS + at + nn]) << 16;
                }
            }
        };
        bool ok = true;
        if (!FULL && nch > 0) {
            const uint32_t z[32] = {};
#pragma unroll 1
            for (int g4 = 0; g4 < P / 64; ++g4) tc::st32(lb + 32 * g4, z);
            tc::wait_st();
            tc::fence_before();
            arrive_w(Lay::S_GO);
        }
        for (int n = 0; FULL && n < nch; ++n) {
            ok = wait_w(Lay::SC_FULL + (n & 1), (n >> 1) & 1);
            if (!ok) break;
            const float4 tot = SM_AT(const float4, sc(n) + SC_TOT);
            const float gam = ex2_approx((tot.x + tot.y) + (tot.z + tot.w));
            arrive_w(Lay::SC_EMPTY + (n & 1));
            if (n > 0) ok = wait_w(Lay::ST_GO, (n - 1) & 1);
            if (!ok) break;
            tc::fence_after();
#pragma unroll 1
            for (int g4 = 0; g4 < P / 64; ++g4) {
                uint32_t r[32];
                if (n == 0) {
                    load_init(g4, r);
                } else {
                    tc::ld32(lb + 32 * g4, r);
                    tc::wait_ld();
                }
                if constexpr (FULL) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c8 = (c0 >> 3) + 4 * g4 + i;
                        const uint32_t at = sb + Lay::H + (c8 >> 3) * Lay::BOX + nn * 128 + (((c8 & 7) ^ (nn & 7)) << 4);
                        SM_AT(uint4, at) = make_uint4(pack_bf16(__uint_as_float(r[8 * i]), __uint_as_float(r[8 * i + 1])),
                                                      pack_bf16(__uint_as_float(r[8 * i + 2]), __uint_as_float(r[8 * i + 3])),
                                                      pack_bf16(__uint_as_float(r[8 * i + 4]), __uint_as_float(r[8 * i + 5])),
                                                      pack_bf16(__uint_as_float(r[8 * i + 6]), __uint_as_float(r[8 * i + 7])));
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(gam * __uint_as_float(r[i]));
                tc::st32(lb + 32 * g4, r);
            }
            tc::wait_st();
            tc::fence_before();
            tc::fence_async_smem();
            arrive_w(Lay::S_GO);
            if constexpr (FULL) arrive_w(Lay::YX_GO);
        }
        const bool write = FULL ? (pc.last && p.fin) : true;
        if (ok && write) {
            if (nch > 0) {
                ok = wait_w(Lay::ST_GO, FULL ? (nch - 1) & 1 : 0);
                tc::fence_after();
            }
#pragma unroll 1
            for (int g4 = 0; ok && g4 < P / 64; ++g4) {
                uint32_t r[32];
                if (nch > 0) {
                    tc::ld32(lb + 32 * g4, r);
                    tc::wait_ld();
                    if (FULL && any_spoilt(r)) {  // stored at the very end, see finish_spoilt
                        spoilt = 1u;
                        continue;
                    }
                } else {
                    load_init(g4, r);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const size_t at = static_cast<size_t>(c0 + 32 * g4 + i) * NS;
                    if constexpr (!FULL)
                        wsp[at] = __uint_as_float(r[i]);
                    else if (!gmem_ok(unit * P * NS + at + nn, 1, st_elems))
                        continue;
                    else if (p.fin_dtype == KDA_DTYPE_FP32)
                        static_cast<float *>(p.fin)[unit * P * NS + at + nn] = __uint_as_float(r[i]);
                    else
                        static_cast<uint16_t *>(p.fin)[unit * P * NS + at + nn] = f2bf_bits(__uint_as_float(r[i]));
                }
            }
        }
        tc::fence_before();
    } else {
        make_wb(warp - Lay::WWB, GROUPS - 1);
    }

    tc::fence_before();
    __syncthreads();
    if constexpr (FULL)
        if (spoilt) finish_spoilt<P, PARTS>(t);
    if (warp == 0) {
        tc::fence_after();
        tc::dealloc(tmem, TMEM_COLS);
    }
#undef SM_AT
}

// Joins the pieces of every (sequence, head): in order, each piece's local state in the workspace is
// replaced by the state that enters the piece, carry <- 2^decay carry + local. Reads and writes the
// workspace once; one thread per four state elements. The chain itself is short; JOIN_BATCH pieces'
// loads are in flight together, as one load's latency per piece is what it would otherwise cost.
constexpr int JOIN_BATCH = 8;
constexpr int JOIN_THREADS = 256;
template <int P>
__global__ void __launch_bounds__(JOIN_THREADS) kda_ssm_join_kernel(const TcParams t)
{
    const ssm::SsmParams &p = t.p;
    constexpr int BLOCKS = P * NS / (4 * JOIN_THREADS);  // CTAs per (sequence, head)
    const int unit = blockIdx.x / BLOCKS, h = unit % p.H, seq = unit / p.H;
    const size_t e = 4 * (static_cast<size_t>(blockIdx.x % BLOCKS) * JOIN_THREADS + threadIdx.x);
    const Span sp = ssm::ssm_span(p, seq);
    if (!sp.ok) return;
    long long base = static_cast<long long>(seq) * t.seg_per_seq;
    if (p.cu) {
        base = 0;
        const int lane = threadIdx.x & 31;
        for (int s0 = 0; s0 < seq; s0 += 32) {
            int n = 0;
            if (s0 + lane < seq) {
                const Span o = ssm::ssm_span(p, s0 + lane);
                n = o.ok ? pieces_of(o.len, t.seg_chunks) : 0;
            }
            base += __reduce_add_sync(0xffffffffu, n);
        }
    }
    const int npieces = pieces_of(sp.len, t.seg_chunks);
    float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
    const size_t u = static_cast<size_t>(unit) * P * NS + e;
    if (p.init) {
        if (p.init_dtype == KDA_DTYPE_FP32) {
            c = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.init) + u);
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.init) + u);
            c = make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
        }
    }
    const float *dec = t.ws + static_cast<size_t>(t.slots) * p.H * P * NS;
    const size_t unit_elems = static_cast<size_t>(P) * NS;
    for (int i0 = 0; i0 < npieces; i0 += JOIN_BATCH) {
        float4 l[JOIN_BATCH];
        float g[JOIN_BATCH];
#pragma unroll
        for (int j = 0; j < JOIN_BATCH; ++j) {
            const long long slot = base + i0 + j;
            // the last piece leaves no local state; overlapping bounds (flagged) have more pieces than there is room for
            if (i0 + j + 1 < npieces && slot < t.slots) {
                const size_t at = static_cast<size_t>(slot) * p.H + h;
                l[j] = __ldcg(reinterpret_cast<const float4 *>(t.ws + at * unit_elems + e));
                g[j] = __ldcg(dec + at);
            }
        }
#pragma unroll
        for (int j = 0; j < JOIN_BATCH; ++j) {
            const long long slot = base + i0 + j;
            if (i0 + j >= npieces || slot >= t.slots) return;
            *reinterpret_cast<float4 *>(t.ws + (static_cast<size_t>(slot) * p.H + h) * unit_elems + e) = c;
            if (i0 + j + 1 < npieces) {
                const float k = ex2_approx(g[j]);
                c = make_float4(fmaf(k, c.x, l[j].x), fmaf(k, c.y, l[j].y), fmaf(k, c.z, l[j].z), fmaf(k, c.w, l[j].w));
            }
        }
    }
}

}  // namespace ssmtc
}  // namespace kda
