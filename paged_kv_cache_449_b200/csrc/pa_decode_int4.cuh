// Decode attention over the 4-bit pools (layout and format: pa_rows.cuh), with
// an optional sliding window and first tokens that stay visible.
//
// With value = zero + scale * code per (token, group of 64 dims), both
// products of attention split into a product over whole-number codes and a
// term of the zeros:
//     q . K_t   = sum_g scale_tg (q_g . code_tg) + zero_tg sum(q_g)
//     sum_t p_t V_td = sum_t (p_t scale_tg) code_td + sum_t p_t zero_tg
// so the tensor cores multiply codes (mma.sync m16n8k16, fp16 operands, fp32
// accumulate; tokens or head dims as M, the heads of a GQA group as N) and
// the scales and zeros cost a few fp32 operations a token and head.
//
// A byte holds the codes a and b of two dims (d and d + 8).  Put at the bottom
// of an fp16 pattern its low four bits are the subnormal a 2^-24, its high four
// 16 b 2^-24, the whole byte (a + 16 b) 2^-24; the tensor cores multiply
// subnormals exactly.  For K the two dims lie along the product's sum: the
// operands are a and 16 b (an AND each, a shift for the upper bytes of the two
// halves), and the sixteenth goes into the query, where it is exact.  For V they
// are rows of the output: the operands are a and a + 16 b, taken
// apart by one subtraction at the end.  (The same for K would take the query
// operand q_d - q_d+8 / 16, which has to be rounded to fp16: outputs were up to
// 5.6e-3 (fp16) and 1.1e-2 (bf16) off for queries of size 32, for one operation
// less in each of the step's 16 words of K, 3% of its instructions.)
//
// Codes are taken about their middle, value = (zero + 7.5 scale) + scale (code
// - 7.5): over many tokens of like weight sum p scale code and sum p zero
// cancel, while the tensor core's sums lose up to 2^-24 of their size at every
// product, always downwards (an error that grew with the square of the
// tokens).  7.5 sum P comes from one more product, with ones, each 16 tokens,
// and leaves the accumulators every fourth step.
//
// Each warp takes steps of 32 tokens (one online-softmax step each) from a
// ring of shared-memory stages of its own, filled by asynchronous 16-byte
// copies of each (block, head) tile, codes and group words; the words lie in
// operand order, so a lane reads its own 16-byte vectors.  (Bulk copies of
// whole tiles, issued by one lane per block, cost about a fifth of the
// kernel's instructions.)
//
// Groups of up to four heads (PACK) fill only half of the product's eight
// columns; there the second half takes the same heads for the other 16 tokens
// of the step (the query operand of a half has zeros in the other's columns), so
// that the softmax and all that is done per score is half the work.
//
// Statistics: fp32 running reference and sum in base 2.  The reference moves
// only when a score exceeds it by 2^8 (one vote a unit instead of a reduction
// and a rescale).  p * scale of V is rounded to fp16 for the product (2^-11,
// where fp32 would take a second product for the remainder), within
// the range of fp16 whatever the scales are: they are taken relative to a
// power of two that moves, like the reference, when a larger scale appears.
// The largest scale lies in [2^5, 2^7) then, so a weight keeps its 11 bits
// down to 2^-19 of it, and below that 2^-30 of the largest scale.
#pragma once

#include "pa_decode.cuh"
#include "pa_rows.cuh"

namespace pa {

// Query group for the fp16 product: each head's row scaled by a 2^shift of its own
// so that its largest magnitude lands in [2^13, 2^14) (up to |q| = 2^114), the
// operands of a 16-dim step being q_d and q_d+8 / 16.  Both are exact (fp16 and
// bf16 elements have 11 and 8 bits), but for elements below 2^-23 of the row's
// largest, which keep 2^-34 of it.  Of heads 2 (lane % 4) + e: sums[c][e]
// the fp32 sum of dims 64 c .., unscaled, shift[e] the scaling.  `raw`: row r's
// dims 16 ks + 2c, + 1 and + 8 of them, as loaded (zero from row `group` on).
template <typename T, int D>
__device__ __forceinline__ void q_operands(uint32_t (&qa)[D / 16][2], float (&sums)[D / 64][2], int (&shift)[2],
                                           const uint32_t (&raw)[D / 16][2], int lane) {
    const int c = lane & 3;
    float f[D / 16][4];
    float mx = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const T* l = reinterpret_cast<const T*>(&raw[ks][0]);
        const T* h = reinterpret_cast<const T*>(&raw[ks][1]);
        f[ks][0] = to_float<T>(l[0]);
        f[ks][1] = to_float<T>(l[1]);
        f[ks][2] = to_float<T>(h[0]);
        f[ks][3] = to_float<T>(h[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(f[ks][e]));
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));   // (of row r)
    // floor(log2(mx)) from the exponent field (a subnormal bf16 maximum counts as 2^-127)
    const int e2 = mx > 0.f ? static_cast<int>((__float_as_uint(mx) >> 23) & 0xff) - 127 : 13;
    const int row_shift = 13 - e2 > 100 ? 100 : (13 - e2 < -100 ? -100 : 13 - e2);
    const float mul = __uint_as_float(static_cast<uint32_t>(127 + row_shift) << 23);   // 2^shift
    shift[0] = __shfl_sync(0xffffffffu, row_shift, 8 * c);
    shift[1] = __shfl_sync(0xffffffffu, row_shift, 8 * c + 4);
#pragma unroll
    for (int ch = 0; ch < D / 64; ++ch) {
        float sum = 0.f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float(&x)[4] = f[4 * ch + m];
            sum += (x[0] + x[1]) + (x[2] + x[3]);
            const __half2 a = __floats2half2_rn(x[0] * mul, x[1] * mul);
            const __half2 b = __floats2half2_rn(x[2] * mul * 0.0625f, x[3] * mul * 0.0625f);
            qa[4 * ch + m][0] = *reinterpret_cast<const uint32_t*>(&a);
            qa[4 * ch + m][1] = *reinterpret_cast<const uint32_t*>(&b);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);   // head r's sum, in the four lanes of row r
        sums[ch][0] = __shfl_sync(0xffffffffu, sum, 8 * c);
        sums[ch][1] = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
    }
}

// D(16x8 f32) = A(16x16 fp16) B(16x8 fp16) + C; not volatile: the compiler may
// place it as it likes.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        const uint32_t (&b)[2], float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// The tokens a decode attends to, in steps of 32: with a window, the steps of
// the first num_sinks tokens and those from position L - window on.
struct VisibleSteps {
    int L, wlo, sinks;   // token t is visible iff t < L and (t >= wlo or t < sinks)
    int first, gap, n;   // n steps: 0 .. first - 1, then first + gap ..
    __device__ __forceinline__ VisibleSteps(int len, int window, int num_sinks) {
        L = len;
        wlo = window > 0 && len > window ? len - window : 0;
        sinks = min(num_sinks, len);
        const int all = (len >> 5) + ((len & 31) != 0), ws = wlo >> 5, ss = (sinks >> 5) + ((sinks & 31) != 0);
        first = ws > ss ? ss : all;
        gap = ws > ss ? ws - ss : 0;
        n = all - gap;
    }
    __device__ __forceinline__ int step(int i) const { return i < first ? i : i + gap; }
    __device__ __forceinline__ bool token(int t) const { return t < L && (t >= wlo || t < sinks); }
    // whether the n tokens from t on are visible, all of them or any
    __device__ __forceinline__ bool whole(int t, int n) const { return L - t >= n && (t >= wlo || sinks - t >= n); }
    __device__ __forceinline__ bool any(int t, int n) const { return t < L && (wlo - t < n || t < sinks); }
};

// Warps an SM holds.  D = 128: 12 of 160 registers (one pass over 64 sequences
// 29.9 us, the 70B long batch 151 us) rather than 16 of 128 (34.9 and 152 us).
template <int D>
constexpr int kInt4Resident = D == 128 ? 12 : 16;
template <int D, int B, int NW, int ST>
struct Int4Smem {
    static constexpr int kTile = int4_tile_bytes(B, D);
    static constexpr int kBlocks = 32 / B;                 // blocks of a step
    static constexpr int kStage = 2 * kBlocks * kTile;     // their K tiles, then their V tiles
    static constexpr int kRing = NW * ST * kStage;
    static constexpr int kMerge = NW * kMaxGroup * (kMergeRow<D> + 2) * 4;   // in the ring's place, after it
    static constexpr int kArea = kRing > kMerge ? kRing : kMerge;
    static constexpr int kTotal = kArea;
    static_assert(kTile % 16 == 0, "copies move 16-byte units");
};

template <typename T, int D, int B, int NW, int ST, bool PACK>
__global__ void __launch_bounds__(NW * 32, kInt4Resident<D> / NW)
    pa_decode_int4_kernel(const __grid_constant__ DecodeParams p) {
    using Sm = Int4Smem<D, B, NW, ST>;
    constexpr int NC = D / 64;                   // groups of a row
    constexpr int kTile = Sm::kTile, kCodes = B * D / 2;
    constexpr int NB = Sm::kBlocks, kSpan = 32 / NB;   // blocks of a step; steps whose ids a warp holds at once
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int last_arrival;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    // The tokens whose scores this lane holds: 8 h + r of the step, h < HN, from
    // token `sub` on (PACK: the lanes of columns 4..7 hold the second 16 tokens)
    constexpr int HN = PACK ? 2 : 4;
    const int sub = PACK ? 16 * (c >> 1) : 0;
    const int part = blockIdx.x, kvh = blockIdx.y;
    int s = blockIdx.z;
    const uint8_t* ring = smem + warp * ST * Sm::kStage;
    wait_for_prior_work();
    if (p.seq_order != nullptr) {
        s = __ldg(p.seq_order + blockIdx.z);
        if (static_cast<unsigned>(s) >= static_cast<unsigned>(p.num_seqs)) {
            if (threadIdx.x == 0 && part == 0 && kvh == 0) flag_error(16 /* PA_DEVERR_SEQ_ORDER */);
            return;
        }
    }
    const int group = p.group;
    int L = p.context_lens[s];
    // Asked for before the length is there: the query, and (without a window,
    // where their places do not depend on it) the first block ids, of which
    // those past the context are dropped below.
    const int32_t* table = p.block_tables + static_cast<long long>(s) * p.max_blocks_per_seq;
    auto early_ids = [&](int span) -> int {
        const long long j = (static_cast<long long>(part) * p.partition_blocks + warp + (span * kSpan + lane / NB) * NW) * NB +
                            lane % NB;
        return p.window == 0 && j < p.max_blocks_per_seq ? __ldg(table + j) : -1;
    };
    const int early0 = early_ids(0), early1 = early_ids(1);
    uint32_t qraw[D / 16][2];
    {
        const int head = PACK ? r & 3 : r;
        const T* row = reinterpret_cast<const T*>(p.q) +
                       (static_cast<long long>(s) * p.num_q_heads + kvh * group + head) * D + 2 * c;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            qraw[ks][0] = head < group ? *reinterpret_cast<const uint32_t*>(row + 16 * ks) : 0u;
            qraw[ks][1] = head < group ? *reinterpret_cast<const uint32_t*>(row + 16 * ks + 8) : 0u;
        }
    }
    if (L < 0 || L > p.context_cap) {
        if (threadIdx.x == 0 && part == 0 && kvh == 0) flag_error(2 /* PA_DEVERR_CONTEXT_LEN */);
        L = L < 0 ? 0 : p.context_cap;
    }
    T* out = reinterpret_cast<T*>(p.out) + (static_cast<long long>(s) * p.num_q_heads + kvh * group) * D;
    const VisibleSteps vis(L, p.window, p.num_sinks);
    const int u0 = part * p.partition_blocks;
    if (u0 >= vis.n) {
        if (part == 0)   // an empty context
            for (int i = threadIdx.x; i < group * D; i += NW * 32) out[i] = from_float<T>(0.f);
        return;
    }
    const int nu = min(vis.n - u0, p.partition_blocks);          // this CTA's steps
    const int n_w = nu > warp ? (nu - warp + NW - 1) / NW : 0;   // this warp's: u0 + warp, + NW, ..
    auto first_token = [&](int i) -> int { return 32 * vis.step(u0 + warp + i * NW); };

    // Block ids, kSpan steps at a time: lane = (step % kSpan) * NB + block of the step
    bool refused = false;   // whether any id so far was (the whole warp knows)
    auto load_ids = [&](int span, int early) -> int {
        const int i = span * kSpan + lane / NB;
        int id = -1;
        bool bad = false;
        if (i < n_w) {
            const int t = first_token(i) + lane % NB * B;
            if (vis.any(t, B)) {
                id = span < 2 && p.window == 0 ? early : __ldg(table + t / B);
                bad = id < 0 || static_cast<long long>(id) >= p.num_blocks;
                if (bad) {
                    flag_error(1 /* PA_DEVERR_BLOCK_ID */);
                    id = -1;
                }
            }
        }
        refused = refused || __any_sync(0xffffffffu, bad);
        return id;
    };
    int ids0 = load_ids(0, early0), ids1 = load_ids(1, early1);
    int span = 0;   // of ids0

    // Copies of step i (of the spans held) into its stage: for each tile the
    // codes, 16 bytes a lane, and the group words of all tiles, 16 bytes a
    // lane too.  A block that is not attended or whose id was refused is left out.
    const uint64_t policy = l2_evict_first_policy();
    const uint32_t stride = static_cast<uint32_t>(p.num_kv_heads) * kTile;
    const uint8_t* kcodes = reinterpret_cast<const uint8_t*>(p.k_cache) + static_cast<long long>(kvh) * kTile + lane * 16;
    const uint8_t* vcodes = reinterpret_cast<const uint8_t*>(p.v_cache) + static_cast<long long>(kvh) * kTile + lane * 16;
    constexpr int PL = B * NC / 4;            // lanes that hold a tile's group words
    const int wt = lane / PL;                 // the tile whose words this lane copies: K's blocks, then V's
    const int word_off = kCodes + lane % PL * 16;
    const uint8_t* wsrc = (wt < NB ? kcodes : vcodes) - lane * 16 + word_off;
    const uint32_t code_dst = smem_u32(ring) + lane * 16, word_dst = smem_u32(ring) + wt * kTile + word_off;
    auto step_id = [&](int i, int block) -> int {   // (a shuffle: the whole warp calls it)
        return __shfl_sync(0xffffffffu, i / kSpan == span ? ids0 : ids1, i % kSpan * NB + block);
    };
    auto at = [&](const uint8_t* base, int id) { return base + static_cast<uint64_t>(static_cast<uint32_t>(id)) * stride; };
    auto issue = [&](int i, uint32_t stage) {   // stage: the stage's offset in the ring
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int id = step_id(i, b);
            if (id >= 0 && (kCodes >= 512 || lane * 16 < kCodes)) {
                copy_codes<kCodes>(code_dst + stage + b * kTile, at(kcodes, id), policy);
                copy_codes<kCodes>(code_dst + stage + (NB + b) * kTile, at(vcodes, id), policy);
            }
        }
        const int id = step_id(i, wt % NB);
        if (id >= 0 && wt < 2 * NB) copy16_async<0>(word_dst + stage, at(wsrc, id), policy);
    };
#pragma unroll
    for (int i = 0; i < ST; ++i) {
        if (i < n_w) issue(i, i * Sm::kStage);
        copy_group_end();
    }

    uint32_t qa[D / 16][2];
    float qsum[NC][2];
    int shift[2];
    q_operands<T, D>(qa, qsum, shift, qraw, lane);
    // PACK: the query operands of the step's first 16 tokens (columns 0..3) and of its second 16 (columns 4..7)
    uint32_t qb[PACK ? D / 16 : 1][2];
    if constexpr (PACK) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qb[ks][e] = r < 4 ? 0u : qa[ks][e];
                qa[ks][e] = r < 4 ? qa[ks][e] : 0u;
            }
    }
    // scores are score_scale 2^(24 - shift) times scale * (the product with codes) + zero * (the sum of q 2^(shift - 24))
    const float code_scale[2] = {ldexpf(p.score_scale, 24 - shift[0]), ldexpf(p.score_scale, 24 - shift[1])};
#pragma unroll
    for (int ch = 0; ch < NC; ++ch)
#pragma unroll
        for (int e = 0; e < 2; ++e) qsum[ch][e] = ldexpf(qsum[ch][e], shift[e] - 24);

    // O^T of codes less 7.5: (d = 16 mt + r, h = 2c), (d, 2c + 1), and that of d plus 16 times that of d + 8, the same heads
    float o[D / 16][4];
    float ps[NC][2];         // sum of P (times 2^-14) that is still to come out of o
    float zo[NC][2];         // sum of p * (zero + 7.5 scale), this lane's tokens
    float m_ref[2] = {0.f, 0.f}, l_run[2] = {0.f, 0.f};
    bool started = false;    // whether a token has been attended: m_ref is a score then
    float v_unit = 0.f;      // scales of V are multiplied by this power of two (0: none seen yet)
    float v_most = 0.f;      // the largest scale that v_unit allows
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) zo[ch][0] = zo[ch][1] = ps[ch][0] = ps[ch][1] = 0.f;

    // The four operand words of 16 tokens (half g of the step) and chunk ch,
    // and the group words of token 8 h + r, from the tiles at `base`.
    auto words = [&](const uint8_t* base, int g, int ch, uint32_t (&w)[4]) {
        if constexpr (B == 8) {   // two blocks of two words; bytes of the two alternate in an operand word
            const uint2 a = *reinterpret_cast<const uint2*>(base + 2 * g * kTile + (ch * 32 + lane) * 8);
            const uint2 b = *reinterpret_cast<const uint2*>(base + (2 * g + 1) * kTile + (ch * 32 + lane) * 8);
            w[0] = __byte_perm(a.x, b.x, 0x6240);
            w[1] = __byte_perm(a.x, b.x, 0x7351);
            w[2] = __byte_perm(a.y, b.y, 0x6240);
            w[3] = __byte_perm(a.y, b.y, 0x7351);
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(
                base + (B == 16 ? g * kTile + (ch * 32 + lane) * 16 : ((g * NC + ch) * 32 + lane) * 16));
            w[0] = a.x;
            w[1] = a.y;
            w[2] = a.z;
            w[3] = a.w;
        }
    };
    auto group_words = [&](const uint8_t* base, int h, uint32_t (&w)[NC]) {
        const int t = sub + 8 * h;
        const uint8_t* at = base + t / B * kTile + kCodes + (t % B + r) * NC * 4;
        if constexpr (NC == 2) {
            const uint2 a = *reinterpret_cast<const uint2*>(at);
            w[0] = a.x;
            w[1] = a.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(at);
        }
    };

    auto centre = [&]() {   // takes 7.5 sum of P out of O
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float(&y)[4] = o[4 * ch + m];
                y[0] = fmaf(-7.5f / 1024.f, ps[ch][0], y[0]);   // (2^-24 / 2^-14)
                y[1] = fmaf(-7.5f / 1024.f, ps[ch][1], y[1]);
                y[2] = fmaf(-127.5f / 1024.f, ps[ch][0], y[2]);
                y[3] = fmaf(-127.5f / 1024.f, ps[ch][1], y[3]);
            }
            ps[ch][0] = ps[ch][1] = 0.f;
        }
    };
    uint32_t stage = 0;   // offset of step i's stage
    for (int i = 0; i < n_w; ++i) {
        if (i / kSpan != span) {
            ++span;
            ids0 = ids1;
            ids1 = load_ids(span + 1, -1);
        }
        copy_groups_wait<ST - 1>();   // this lane's copies of the step; then every lane's
        __syncwarp();
        const uint8_t* kbase = ring + stage;
        const uint8_t* vbase = kbase + NB * kTile;
        const int t0 = first_token(i);
        const bool whole = vis.whole(t0, 32) && !refused;

        // S^T of codes, per group of dims; scores x[2h], x[2h + 1] of this lane's token h and two heads
        // relative to the softmax's reference
        float x[2 * HN];
#pragma unroll
        for (int e = 0; e < 2 * HN; ++e) x[e] = 0.f;
        float sc[HN / 2][NC][4];
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            uint32_t wa[4], wb[4];
            words(kbase, 0, ch, wa);
            words(kbase, 1, ch, wb);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {   // tokens r: bytes 0 and 2; r + 8: bytes 1 and 3
                    const bool first = m == 0 && (!PACK || g == 0);
                    const uint32_t w = g ? wb[m] : wa[m];
                    const uint32_t f = w >> 8;
                    float(&y)[4] = sc[PACK ? 0 : g][ch];
                    mma_f16(y, w & 0x000f000fu, f & 0x000f000fu, w & 0x00f000f0u, f & 0x00f000f0u, PACK && g ? qb[PACK ? 4 * ch + m : 0] : qa[4 * ch + m],
                            first ? 0.f : y[0], first ? 0.f : y[1], first ? 0.f : y[2], first ? 0.f : y[3]);
                }
            }
        }
        float vs[HN][NC], vz[HN][NC];   // V's scales, and the values of code 7.5
#pragma unroll
        for (int h = 0; h < HN; ++h) {
            uint32_t kw[NC], vw[NC];
            group_words(kbase, h, kw);
            group_words(vbase, h, vw);
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) {
                const float ks = __uint_as_float(kw[ch] << 16);
                const float kz = __uint_as_float(kw[ch] & 0xffff0000u);
                const float(&q)[4] = sc[h / 2][ch];
                x[2 * h] = fmaf(ks, q[2 * (h & 1)], fmaf(kz, qsum[ch][0], x[2 * h]));
                x[2 * h + 1] = fmaf(ks, q[2 * (h & 1) + 1], fmaf(kz, qsum[ch][1], x[2 * h + 1]));
                vs[h][ch] = __uint_as_float(vw[ch] << 16);
                vz[h][ch] = fmaf(7.5f, vs[h][ch], __uint_as_float(vw[ch] & 0xffff0000u));
            }
            x[2 * h] = fmaf(x[2 * h], code_scale[0], -m_ref[0]);
            x[2 * h + 1] = fmaf(x[2 * h + 1], code_scale[1], -m_ref[1]);
        }
        if (!whole) {   // tokens that are not attended, or whose block id was refused: whatever lies there is not used
#pragma unroll
            for (int h = 0; h < HN; ++h) {
                const int t = sub + 8 * h;
                if (!(step_id(i, t / B) >= 0 && vis.token(t0 + t + r))) {
                    x[2 * h] = x[2 * h + 1] = kNegInf;
#pragma unroll
                    for (int ch = 0; ch < NC; ++ch) vs[h][ch] = vz[h][ch] = 0.f;
                }
            }
        }
        // the reference of the softmax and the unit of V's scales, moved when they have to be
        float mx0 = x[0], mx1 = x[1], sm = 0.f;
#pragma unroll
        for (int h = 0; h < HN; ++h) {
            mx0 = fmaxf(mx0, x[2 * h]);
            mx1 = fmaxf(mx1, x[2 * h + 1]);
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) sm = fmaxf(sm, vs[h][ch]);
        }
        if (__any_sync(0xffffffffu, mx0 > 8.f || mx1 > 8.f || sm > v_most) || !started) {
            float n0 = mx0, n1 = mx1;   // by how much the references rise
#pragma unroll
            for (int off = PACK ? 2 : 4; off < 32; off <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
                n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
            }
            if (sm == INFINITY) {   // a group that is not finite: its output is not, and the unit is the others'
                sm = 0.f;
#pragma unroll
                for (int h = 0; h < HN; ++h)
#pragma unroll
                    for (int ch = 0; ch < NC; ++ch) sm = vs[h][ch] < INFINITY ? fmaxf(sm, vs[h][ch]) : sm;
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) sm = fmaxf(sm, __shfl_xor_sync(0xffffffffu, sm, off));
            const bool any = __any_sync(0xffffffffu, n0 != kNegInf);   // (a step masks all heads alike)
            n0 = !any ? 0.f : (started ? fmaxf(n0, 0.f) : n0);
            n1 = !any ? 0.f : (started ? fmaxf(n1, 0.f) : n1);
            // (before the start there is nothing to rescale, and n may be far below zero)
            const float a0 = started ? exp2_approx(-n0) : 1.f, a1 = started ? exp2_approx(-n1) : 1.f;
            started = started || any;
            m_ref[0] += n0;
            m_ref[1] += n1;
#pragma unroll
            for (int h = 0; h < HN; ++h) {
                x[2 * h] -= n0;
                x[2 * h + 1] -= n1;
            }
            float vu = 1.f;
            if (sm > v_most) {   // (scales are bf16: below 2^128)
                const int e = static_cast<int>((__float_as_uint(sm) >> 23) & 0xff) - 127;   // sm < 2^(e + 1)
                int up = 5 - e;                                                             // p * scale <= 2^8 2^7
                up = up > 126 ? 126 : up;
                const float unit = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                vu = v_unit > 0.f ? unit / v_unit : 1.f;
                v_unit = unit;
                v_most = __uint_as_float(static_cast<uint32_t>(127 + (7 - up > 127 ? 127 : 7 - up)) << 23);
            }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                o[mt][0] *= a0 * vu;
                o[mt][1] *= a1 * vu;
                o[mt][2] *= a0 * vu;
                o[mt][3] *= a1 * vu;
            }
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) {
                zo[ch][0] *= a0;
                zo[ch][1] *= a1;
                ps[ch][0] *= a0 * vu;
                ps[ch][1] *= a1 * vu;
            }
            l_run[0] *= a0;
            l_run[1] *= a1;
        }
#pragma unroll
        for (int e = 0; e < 2 * HN; ++e) {   // x becomes p
            x[e] = exp2_approx(x[e]);
            l_run[e & 1] += x[e];
        }
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            uint32_t pb[2][2];   // P^T as the B operand, tokens 16 g + 8 e ..
#pragma unroll
            for (int h = 0; h < HN; ++h) {
                zo[ch][0] = fmaf(x[2 * h], vz[h][ch], zo[ch][0]);
                zo[ch][1] = fmaf(x[2 * h + 1], vz[h][ch], zo[ch][1]);
                const float sv = vs[h][ch] * v_unit;
                pb[h / 2][h % 2] = movmatrix_trans(Mma<__half>::pack(x[2 * h] * sv, x[2 * h + 1] * sv));
            }
            uint32_t wa[4], wb[4];
            words(vbase, 0, ch, wa);
            words(vbase, 1, ch, wb);
            // the codes' mean part: 7.5 sum of P (as rounded), the same in every row.
            // The ones are 2^-14, a normal number: the tensor core aligns a
            // product by its operands' exponents, so one with the subnormal 2^-24
            // keeps ten bits less of the sum (and 7.5 times that is lost: 1.6e-3
            // of a 32k context's output).
            float mean[4];
            mma_f16(mean, 0x04000400u, 0x04000400u, 0x04000400u, 0x04000400u, pb[0], ps[ch][0], ps[ch][1], 0.f, 0.f);
            if constexpr (PACK) {   // (both halves of the step in one product) then each half's columns alone
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    pb[1][e] = r < 4 ? 0u : pb[0][e];
                    pb[0][e] = r < 4 ? pb[0][e] : 0u;
                }
            } else {
                mma_f16(mean, 0x04000400u, 0x04000400u, 0x04000400u, 0x04000400u, pb[1], mean[0], mean[1], mean[2], mean[3]);
            }
            ps[ch][0] = mean[0];
            ps[ch][1] = mean[1];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float(&y)[4] = o[4 * ch + m];
#pragma unroll
                for (int g = 0; g < 2; ++g) {   // tokens 2c, 2c + 1: bytes 0 and 2; + 8: bytes 1 and 3
                    const uint32_t w = g ? wb[m] : wa[m];
                    const uint32_t e = w & 0x00ff00ffu, f = __byte_perm(w, 0u, 0x4341);
                    mma_f16(y, e & 0x000f000fu, e, f & 0x000f000fu, f, pb[g], y[0], y[1], y[2], y[3]);
                }
            }
        }
        if ((i & 3) == 3) centre();
        __syncwarp();   // every lane has read the stage
        if (i + ST < n_w) issue(i + ST, stage);
        copy_group_end();
        stage = stage == (ST - 1) * Sm::kStage ? 0u : stage + Sm::kStage;
    }
    centre();
    copy_groups_wait<0>();
    __syncthreads();   // (the ring is free now)

    // ---- this warp's state in true units, then the warps' merge
    if constexpr (PACK) {   // the two halves of the steps
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][e] += __shfl_xor_sync(0xffffffffu, o[mt][e], 2);
    }
    float* mo = reinterpret_cast<float*>(smem);
    float* mml = mo + NW * kMaxGroup * kMergeRow<D>;
    // 2^24 / unit, in two factors: the quotient is infinite for units below 2^-104
    const float back = v_unit > 0.f ? 1.f / v_unit : 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = PACK ? 2 : 4; off < 32; off <<= 1) {
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], off);
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) zo[ch][e] += __shfl_xor_sync(0xffffffffu, zo[ch][e], off);
        }
        const int h = 2 * c + e;
        if (h < group) {
            float* row = mo + (warp * kMaxGroup + h) * kMergeRow<D>;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                row[16 * mt + r] = fmaf(o[mt][e] * 16777216.f, back, zo[mt / 4][e]);
                row[16 * mt + 8 + r] = fmaf((o[mt][2 + e] - o[mt][e]) * 1048576.f, back, zo[mt / 4][e]);
            }
            if (r == 0) {
                mml[(warp * kMaxGroup + h) * 2] = started ? m_ref[e] : kNegInf;
                mml[(warp * kMaxGroup + h) * 2 + 1] = l_run[e];
            }
        }
    }
    __syncthreads();
    const int num_parts = (vis.n + p.partition_blocks - 1) / p.partition_blocks;
    for (int v = threadIdx.x; v < group * (D / 4); v += NW * 32) {   // four dims of a head each
        const int h = v / (D / 4), d = v % (D / 4) * 4;
        float m[NW], M = kNegInf;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, m[w] = mml[(w * kMaxGroup + h) * 2]);
        const float top = M == kNegInf ? 0.f : M;
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
        float den = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float wt = exp2_approx(m[w] - top);
            const float4 x = *reinterpret_cast<const float4*>(mo + (w * kMaxGroup + h) * kMergeRow<D> + d);
            num.x = fmaf(wt, x.x, num.x);
            num.y = fmaf(wt, x.y, num.y);
            num.z = fmaf(wt, x.z, num.z);
            num.w = fmaf(wt, x.w, num.w);
            den = fmaf(wt, mml[(w * kMaxGroup + h) * 2 + 1], den);
        }
        if (num_parts > 1) {
            const long long slot = (static_cast<long long>(s) * p.num_q_heads + kvh * group + h) * p.num_partitions + part;
            *reinterpret_cast<float4*>(p.part_acc + slot * D + d) = num;
            if (d == 0) *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(M, den);
        } else {
            store4<T>(out + h * D + d, num, den > 0.f ? 1.f / den : 0.f);
        }
    }
    if (num_parts > 1) {   // the CTA that brings a (sequence, kv head)'s last partition merges them
        // (the barrier orders the CTA's writes before thread 0's fence, which covers them)
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            last_arrival = atomicAdd(p.counters + static_cast<long long>(s) * p.num_kv_heads + kvh, 1) == num_parts - 1;
        }
        __syncthreads();
        if (last_arrival) {
            __threadfence();
            merge_partials<T, D, true, NW * 32>(p, s, kvh, num_parts, reinterpret_cast<float*>(smem), Sm::kArea / 4);
            if (threadIdx.x == 0) p.counters[static_cast<long long>(s) * p.num_kv_heads + kvh] = 0;
        }
    }
}

}  // namespace pa
