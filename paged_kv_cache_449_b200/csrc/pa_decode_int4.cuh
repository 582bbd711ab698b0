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
// A code becomes an fp16 operand with one AND: four bits placed at the bottom
// of an fp16 pattern are the subnormal code * 2^-24, four bits one nibble
// higher code * 2^-20; the tensor cores multiply subnormals exactly.  The
// factor 16 between the two is taken back where it is free: for K (nibble =
// upper half of a 16-dim step) in the query operand, for V (nibble = upper
// eight dims of a 16-dim tile) in the output rows.  A word of a tile is then a
// whole operand of one MMA in five operations.
//
// The words lie in HBM in operand order, so a lane loads its own 16-byte
// vectors straight into registers: no staging in shared memory, no barriers,
// and the next units' loads stay in flight under the present one's arithmetic.
//
// Statistics: fp32 running reference and sum in base 2.  The reference moves
// only when a score exceeds it by 2^8 (one vote a unit instead of a reduction
// and a rescale).  p * scale of V is rounded to fp16 for the product, within
// the range of fp16 whatever the scales are: they are taken relative to a
// power of two that moves, like the reference, when a larger scale appears.
#pragma once

#include "pa_decode.cuh"
#include "pa_rows.cuh"

namespace pa {

// Query group for the fp16 product: rows scaled by 2^shift so that the largest
// magnitude lands in [2^13, 2^14) (exact for every element within 2^-23 of it),
// the upper eight dims of each 16-dim step by a further 1/16.  sums[c][e]: the
// fp32 sum of dims 64 c .. of heads 2 (lane % 4) + e, unscaled.
template <typename T, int D>
__device__ __forceinline__ int load_q_int4(uint32_t (&qa)[D / 16][2], float (&sums)[D / 64][2], const T* q_rows,
                                           int group, int lane) {
    const int r = lane >> 2, c = lane & 3;
    float f[D / 16][4];
    float mx = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t lo = 0u, hi = 0u;
        if (r < group) {
            lo = *reinterpret_cast<const uint32_t*>(q_rows + r * D + ks * 16 + 2 * c);
            hi = *reinterpret_cast<const uint32_t*>(q_rows + r * D + ks * 16 + 8 + 2 * c);
        }
        const T* l = reinterpret_cast<const T*>(&lo);
        const T* h = reinterpret_cast<const T*>(&hi);
        f[ks][0] = to_float<T>(l[0]);
        f[ks][1] = to_float<T>(l[1]);
        f[ks][2] = to_float<T>(h[0]);
        f[ks][3] = to_float<T>(h[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(f[ks][e]));
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    // floor(log2(mx)) from the exponent field (a subnormal bf16 maximum counts as 2^-127)
    const int e2 = mx > 0.f ? static_cast<int>((__float_as_uint(mx) >> 23) & 0xff) - 127 : 13;
    int shift = 13 - e2;
    shift = shift > 100 ? 100 : (shift < -100 ? -100 : shift);
    const float mul = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);   // 2^shift
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
    return shift;
}

// Loads of data read once: past L1, first out of L2.
__device__ __forceinline__ uint4 ldg_stream16(const uint8_t* p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
    return v;
}
__device__ __forceinline__ uint2 ldg_stream8(const uint8_t* p, uint64_t policy) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v2.u32 {%0,%1}, [%2], %3;"
                 : "=r"(v.x), "=r"(v.y)
                 : "l"(p), "l"(policy));
    return v;
}
__device__ __forceinline__ uint32_t ldg_stream4(const uint8_t* p, uint64_t policy) {
    uint32_t v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.u32 %0, [%1], %2;" : "=r"(v) : "l"(p), "l"(policy));
    return v;
}

// The tokens a decode attends to, in units of 16: with a window, the units of
// the first num_sinks tokens and those from position L - window on.
struct VisibleUnits {
    int L, wlo, sinks;   // token t is visible iff t < L and (t >= wlo or t < sinks)
    int first, gap, n;   // n units: 0 .. first - 1, then first + gap ..
    __device__ __forceinline__ VisibleUnits(int len, int window, int num_sinks) {
        L = len;
        wlo = window > 0 && len > window ? len - window : 0;
        sinks = min(num_sinks, len);
        const int units = (len + 15) >> 4, wu = wlo >> 4, su = (sinks + 15) >> 4;
        first = wu > su ? su : units;
        gap = wu > su ? wu - su : 0;
        n = units - gap;
    }
    __device__ __forceinline__ int unit(int i) const { return i < first ? i : i + gap; }
    __device__ __forceinline__ bool token(int t) const { return t < L && (t >= wlo || t < sinks); }
    // whether [t, t + 16) is visible whole
    __device__ __forceinline__ bool whole(int t) const { return t + 16 <= L && (t >= wlo || t + 16 <= sinks); }
    // whether any of [t, t + n) is visible
    __device__ __forceinline__ bool any(int t, int n) const { return t < L && (t + n > wlo || t < sinks); }
};

// One unit's words: K and V codes (per 64 dims; 8-token blocks: two words of
// the unit's first block, two of its second) and the group words of tokens r
// and r + 8.
template <int D>
struct UnitInt4 {
    uint4 k[D / 64], v[D / 64];
    uint32_t kw[2][D / 64], vw[2][D / 64];
    int ok;   // bit 0, 1: the block of tokens 0..7, 8..15 of the unit may be read
};

template <typename T, int D, int B, int NW>
__global__ void __launch_bounds__(NW * 32, (D == 64 ? 16 : 12) / NW)
    pa_decode_int4_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int NC = D / 64;                   // groups of a row
    constexpr int kTile = int4_tile_bytes(B, D);
    constexpr int kCodes = B * D / 2;
    constexpr int kDepth = 2;                    // units loaded ahead
    __shared__ float mo[NW * kMaxGroup * kMergeRow<D>];
    __shared__ float mml[NW * kMaxGroup * 2];
    __shared__ int last_arrival;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    const int part = blockIdx.x, kvh = blockIdx.y;
    int s = blockIdx.z;
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
    if (L < 0 || L > p.context_cap) {
        if (threadIdx.x == 0 && part == 0 && kvh == 0) flag_error(2 /* PA_DEVERR_CONTEXT_LEN */);
        L = L < 0 ? 0 : p.context_cap;
    }
    T* out = reinterpret_cast<T*>(p.out) + (static_cast<long long>(s) * p.num_q_heads + kvh * group) * D;
    const VisibleUnits vis(L, p.window, p.num_sinks);
    const int u0 = part * p.partition_blocks;
    if (u0 >= vis.n) {
        if (part == 0)   // an empty context
            for (int i = threadIdx.x; i < group * D; i += NW * 32) out[i] = from_float<T>(0.f);
        return;
    }
    const int nu = min(vis.n - u0, p.partition_blocks);          // this CTA's units
    const int n_w = nu > warp ? (nu - warp + NW - 1) / NW : 0;   // this warp's: u0 + warp, + NW, ..

    const int32_t* table = p.block_tables + static_cast<long long>(s) * p.max_blocks_per_seq;
    // ids of the blocks under this warp's unit i, 32 units at a time, lane = i % 32
    auto load_id = [&](int i, int half) -> int {
        if (i >= n_w) return -1;
        const int t = 16 * vis.unit(u0 + warp + i * NW) + (B == 8 ? 8 * half : 0);
        if (!vis.any(t, B == 8 ? 8 : 16)) return -1;
        const int id = __ldg(table + t / B);
        if (id >= 0 && static_cast<long long>(id) < p.num_blocks) return id;
        flag_error(1 /* PA_DEVERR_BLOCK_ID */);
        return -1;
    };
    int ids[2], ids8[2] = {-1, -1};   // two windows of 32 units (8-token blocks: and the units' second blocks)
    ids[0] = load_id(lane, 0);
    ids[1] = load_id(32 + lane, 0);
    if constexpr (B == 8) {
        ids8[0] = load_id(lane, 1);
        ids8[1] = load_id(32 + lane, 1);
    }
    int window0 = 0;   // first unit of ids[0]

    const uint64_t policy = l2_evict_first_policy();
    const uint8_t* kpool = reinterpret_cast<const uint8_t*>(p.k_cache);
    const uint8_t* vpool = reinterpret_cast<const uint8_t*>(p.v_cache);
    auto fetch = [&](UnitInt4<D>& f, int i) {   // warp-uniform i
        const int w = (i - window0) >> 5;
        const int id = __shfl_sync(0xffffffffu, w ? ids[1] : ids[0], i & 31);
        if constexpr (B == 8) {
            const int id8 = __shfl_sync(0xffffffffu, w ? ids8[1] : ids8[0], i & 31);
            f.ok = (id >= 0 ? 1 : 0) | (id8 >= 0 ? 2 : 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int b = h ? id8 : id;
                const long long at = (static_cast<long long>(b < 0 ? 0 : b) * p.num_kv_heads + kvh) * kTile;
#pragma unroll
                for (int ch = 0; ch < NC; ++ch) {
                    uint2 k = make_uint2(0u, 0u), v = make_uint2(0u, 0u);
                    f.kw[h][ch] = f.vw[h][ch] = 0u;
                    if (b >= 0) {
                        k = ldg_stream8(kpool + at + (ch * 32 + lane) * 8, policy);
                        v = ldg_stream8(vpool + at + (ch * 32 + lane) * 8, policy);
                        f.kw[h][ch] = ldg_stream4(kpool + at + kCodes + (r * NC + ch) * 4, policy);
                        f.vw[h][ch] = ldg_stream4(vpool + at + kCodes + (r * NC + ch) * 4, policy);
                    }
                    if (h == 0) {
                        f.k[ch].x = k.x; f.k[ch].y = k.y; f.v[ch].x = v.x; f.v[ch].y = v.y;
                    } else {
                        f.k[ch].z = k.x; f.k[ch].w = k.y; f.v[ch].z = v.x; f.v[ch].w = v.y;
                    }
                }
            }
        } else {
            f.ok = id >= 0 ? 3 : 0;
            if (id >= 0) {
                const int tg = B == 32 ? (vis.unit(u0 + warp + i * NW) & 1) : 0;
                const long long at = (static_cast<long long>(id) * p.num_kv_heads + kvh) * kTile;
#pragma unroll
                for (int ch = 0; ch < NC; ++ch) {
                    f.k[ch] = ldg_stream16(kpool + at + ((tg * NC + ch) * 32 + lane) * 16, policy);
                    f.v[ch] = ldg_stream16(vpool + at + ((tg * NC + ch) * 32 + lane) * 16, policy);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const long long w0 = at + kCodes + (16 * tg + r + 8 * h) * NC * 4;
                    if constexpr (NC == 2) {
                        const uint2 k = ldg_stream8(kpool + w0, policy), v = ldg_stream8(vpool + w0, policy);
                        f.kw[h][0] = k.x; f.kw[h][1] = k.y; f.vw[h][0] = v.x; f.vw[h][1] = v.y;
                    } else {
                        f.kw[h][0] = ldg_stream4(kpool + w0, policy);
                        f.vw[h][0] = ldg_stream4(vpool + w0, policy);
                    }
                }
            }
        }
    };

    UnitInt4<D> f[kDepth];
#pragma unroll
    for (int k = 0; k < kDepth; ++k)
        if (k < n_w) fetch(f[k], k);

    uint32_t qa[D / 16][2];
    float qsum[NC][2];
    const T* qrows = reinterpret_cast<const T*>(p.q) + (static_cast<long long>(s) * p.num_q_heads + kvh * group) * D;
    const int shift = load_q_int4<T, D>(qa, qsum, qrows, group, lane);
    const float code_scale = ldexpf(p.score_scale, 24 - shift);
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) {
        qsum[ch][0] *= p.score_scale;
        qsum[ch][1] *= p.score_scale;
    }

    float o[D / 16][4];      // O^T of codes: (d = 16 mt + r, h = 2c), (d, 2c + 1), (d + 8, 2c) x 16, (d + 8, 2c + 1) x 16
    float zo[NC][2];         // sum of p * zero, this lane's tokens
    float m_ref[2] = {kNegInf, kNegInf}, l_run[2] = {0.f, 0.f};
    float v_unit = 0.f;      // scales of V are multiplied by this power of two (0: none seen yet)
    float v_most = 0.f;      // the largest scale that v_unit allows
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) zo[ch][0] = zo[ch][1] = 0.f;

    // the operand words of MMA m of chunk ch, from the unit's words
    auto word = [&](const uint4& x, int m) -> uint32_t {
        if constexpr (B == 8) {
            const uint32_t a = m < 2 ? x.x : x.y, b = m < 2 ? x.z : x.w;
            return __byte_perm(a, b, (m & 1) ? 0x7351 : 0x6240);
        } else {
            return m == 0 ? x.x : (m == 1 ? x.y : (m == 2 ? x.z : x.w));
        }
    };

    auto compute = [&](const UnitInt4<D>& u, int i) {
        // S^T of codes, per group of dims
        float sc[NC][4];
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            sc[ch][0] = sc[ch][1] = sc[ch][2] = sc[ch][3] = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t x = word(u.k[ch], m), y = x >> 8;
                Mma<__half>::k16(sc[ch], x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u, y & 0x00f000f0u,
                                 qa[4 * ch + m][0], qa[4 * ch + m][1]);
            }
        }
        float x[4] = {0.f, 0.f, 0.f, 0.f};   // scores: (token r, head 2c), (r, 2c + 1), (r + 8, 2c), (r + 8, 2c + 1)
        float vs[2][NC], vz[2][NC];
        const int t0 = 16 * vis.unit(u0 + warp + i * NW) + r;
        const bool whole = u.ok == 3 && vis.whole(t0 - r);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) {
                const float ks = __uint_as_float(u.kw[h][ch] << 16) * code_scale;
                const float kz = __uint_as_float(u.kw[h][ch] & 0xffff0000u);
                x[2 * h] = fmaf(ks, sc[ch][2 * h], fmaf(kz, qsum[ch][0], x[2 * h]));
                x[2 * h + 1] = fmaf(ks, sc[ch][2 * h + 1], fmaf(kz, qsum[ch][1], x[2 * h + 1]));
                vs[h][ch] = __uint_as_float(u.vw[h][ch] << 16);
                vz[h][ch] = __uint_as_float(u.vw[h][ch] & 0xffff0000u);
            }
            if (!whole) {   // tokens that are not attended, or whose block id was refused: whatever lies there is not used
                if (!(((u.ok >> h) & 1) && vis.token(t0 + 8 * h))) {
                    x[2 * h] = x[2 * h + 1] = kNegInf;
#pragma unroll
                    for (int ch = 0; ch < NC; ++ch) vs[h][ch] = vz[h][ch] = 0.f;
                }
            }
        }
        // the reference of the softmax and the unit of V's scales, moved when they have to be
        const float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
        float sm = fmaxf(vs[0][0], vs[1][0]);
        if constexpr (NC == 2) sm = fmaxf(sm, fmaxf(vs[0][1], vs[1][1]));
        if (__any_sync(0xffffffffu, mx0 > m_ref[0] + 8.f || mx1 > m_ref[1] + 8.f || sm > v_most)) {
            float n0 = fmaxf(m_ref[0], mx0), n1 = fmaxf(m_ref[1], mx1);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
                n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) sm = fmaxf(sm, __shfl_xor_sync(0xffffffffu, sm, off));
            const float a0 = n0 == kNegInf ? 1.f : exp2_approx(m_ref[0] - n0);
            const float a1 = n1 == kNegInf ? 1.f : exp2_approx(m_ref[1] - n1);
            m_ref[0] = n0;
            m_ref[1] = n1;
            float vu = 1.f;
            if (sm > v_most) {   // (scales are bf16: at most 2^128; an infinite one makes the output NaN)
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
            }
            l_run[0] *= a0;
            l_run[1] *= a1;
        }
        const float mu0 = m_ref[0] == kNegInf ? 0.f : m_ref[0], mu1 = m_ref[1] == kNegInf ? 0.f : m_ref[1];
        const float p0 = exp2_approx(x[0] - mu0), p1 = exp2_approx(x[1] - mu1);
        const float p2 = exp2_approx(x[2] - mu0), p3 = exp2_approx(x[3] - mu1);
        l_run[0] += p0 + p2;
        l_run[1] += p1 + p3;
#pragma unroll
        for (int ch = 0; ch < NC; ++ch) {
            zo[ch][0] = fmaf(p0, vz[0][ch], fmaf(p2, vz[1][ch], zo[ch][0]));
            zo[ch][1] = fmaf(p1, vz[0][ch], fmaf(p3, vz[1][ch], zo[ch][1]));
            const float s0 = vs[0][ch] * v_unit, s1 = vs[1][ch] * v_unit;
            const uint32_t b0 = movmatrix_trans(Mma<__half>::pack(p0 * s0, p1 * s0));
            const uint32_t b1 = movmatrix_trans(Mma<__half>::pack(p2 * s1, p3 * s1));
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t w = word(u.v[ch], m), y = w >> 8;
                Mma<__half>::k16(o[4 * ch + m], w & 0x000f000fu, w & 0x00f000f0u, y & 0x000f000fu, y & 0x00f000f0u,
                                 b0, b1);
            }
        }
    };

    for (int i = 0; i < n_w; i += kDepth) {
        if (i - window0 >= 32) {   // (kDepth divides 32: a window starts at an i of this loop)
            window0 += 32;
            ids[0] = ids[1];
            ids[1] = load_id(window0 + 32 + lane, 0);
            if constexpr (B == 8) {
                ids8[0] = ids8[1];
                ids8[1] = load_id(window0 + 32 + lane, 1);
            }
        }
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            if (i + k < n_w) {
                compute(f[k], i + k);
                if (i + k + kDepth < n_w) fetch(f[k], i + k + kDepth);
            }
        }
    }

    // ---- this warp's state in true units, then the warps' merge
    const float back = v_unit > 0.f ? 16777216.f / v_unit : 0.f;   // 2^24 / unit
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], off);
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) zo[ch][e] += __shfl_xor_sync(0xffffffffu, zo[ch][e], off);
        }
        const int h = 2 * c + e;
        if (h < group) {
            float* row = mo + (warp * kMaxGroup + h) * kMergeRow<D>;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                row[16 * mt + r] = fmaf(o[mt][e], back, zo[mt / 4][e]);
                row[16 * mt + 8 + r] = fmaf(o[mt][2 + e], back * 0.0625f, zo[mt / 4][e]);
            }
            if (r == 0) {
                mml[(warp * kMaxGroup + h) * 2] = m_ref[e];
                mml[(warp * kMaxGroup + h) * 2 + 1] = l_run[e];
            }
        }
    }
    __syncthreads();
    const int num_parts = (vis.n + p.partition_blocks - 1) / p.partition_blocks;
    for (int idx = threadIdx.x; idx < group * D; idx += NW * 32) {
        const int h = idx / D, d = idx - h * D;
        float M = kNegInf;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, mml[(w * kMaxGroup + h) * 2]);
        float num = 0.f, den = 0.f;
        if (M != kNegInf) {
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float wt = exp2_approx(mml[(w * kMaxGroup + h) * 2] - M);
                num = fmaf(wt, mo[(w * kMaxGroup + h) * kMergeRow<D> + d], num);
                den = fmaf(wt, mml[(w * kMaxGroup + h) * 2 + 1], den);
            }
        }
        if (num_parts > 1) {
            const long long slot = (static_cast<long long>(s) * p.num_q_heads + kvh * group + h) * p.num_partitions + part;
            p.part_acc[slot * D + d] = num;
            if (d == 0) {
                p.part_ml[slot * 2] = M;
                p.part_ml[slot * 2 + 1] = den;
            }
        } else {
            out[idx] = from_float<T>(den > 0.f ? num / den : 0.f);
        }
    }
    if (num_parts > 1) {   // the CTA that brings a (sequence, kv head)'s last partition merges them
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0)
            last_arrival = atomicAdd(p.counters + static_cast<long long>(s) * p.num_kv_heads + kvh, 1) == num_parts - 1;
        __syncthreads();
        if (last_arrival) {
            __threadfence();
            merge_partitions_cta<T, D, true, NW * 32>(p, s, kvh, num_parts);
            if (threadIdx.x == 0) p.counters[static_cast<long long>(s) * p.num_kv_heads + kvh] = 0;
        }
    }
}

}  // namespace pa
