// Rows of new tokens held in registers and written into a paged pool: the
// part that the cache writes share, whatever the pool's element type
// ("从源码剖析 vLLM 的显存管理与连续批处理" §2.1, BlockTable.append_token).
//
// A head's row of D elements lies in D / E consecutive lanes of a warp, E = 16
// bytes / element size elements each (one 16-byte vector), widened to fp32.
//
// The 4-bit pools.  The 64 dims of a group (of one token and kv head) share a
// scale and a zero:
//     zero  = the group's minimum rounded down to bf16
//     scale = (maximum - zero) / 15 rounded up to bf16 (0 if that is 0, else at least 2^-126)
//     code  = (x - zero) / scale rounded to the nearest whole number, ties to even, in 0..15
//     value = zero + scale * code
// (every step in fp32).  The roundings outwards keep the whole group inside
// [zero, zero + 15 scale], so no value is clipped by more than fp32's own
// rounding; bf16 covers every input type's range, where fp16 would not.
// Groups of 64 dims cost 4 bytes per 32 bytes of codes.
//
// One (block, kv head) tile is B * D / 2 bytes of codes, then B * D / 64 words
// (token, group: scale in the low half, zero in the high half).  The codes
// lie in the order of the 16-bit tensor-core operand that the decode makes of
// them: for each 16 tokens and 64 dims, 32 lanes x 4 words; a word is one
// lane's share of a 16 x 16 operand tile.  A byte holds dims d (low nibble)
// and d + 8 of one token, so that no two tokens share a byte and a write
// needs no read.  (8-token blocks: 32 lanes x 2 words for 8 tokens, a word
// for two such tiles' halves.)
#pragma once

#include "pa_device.cuh"
#include "pa_e4m3.cuh"

namespace pa {

enum class Pool { kNative, kE4m3, kInt4 };

constexpr int kInt4Group = 64;

// Bytes of a 4-bit (block, kv head) tile.
__host__ __device__ constexpr int int4_tile_bytes(int B, int D) { return B * D / 2 + B * (D / kInt4Group) * 4; }

// Offset in a tile of the byte that holds dims d and d + 8 (d % 16 < 8) of
// token t.  K: the operand's rows are tokens, its columns dims; V: the
// operand is V^T.
__device__ __forceinline__ int int4_code_byte(bool value, int B, int D, int t, int d) {
    const int chunk = d >> 6, m = (d >> 4) & 3, e = d & 7, u = t & 7;
    const int lane = value ? e * 4 + (u >> 1) : u * 4 + (e >> 1);
    const int odd = value ? (u & 1) : (e & 1);
    if (B == 8) return (chunk * 32 + lane) * 8 + (m >> 1) * 4 + (m & 1) + 2 * odd;
    return (((t >> 4) * (D >> 6) + chunk) * 32 + lane) * 16 + m * 4 + ((t >> 3) & 1) + 2 * odd;
}

// One 16-byte vector of T, widened.
template <typename T>
struct Vec {
    static constexpr int E = 16 / static_cast<int>(sizeof(T));
    float f[E];
    __device__ __forceinline__ void load(const T* p) { widen(*reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void widen(const uint4& w) {
        const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = to_float<T>(e[i]);
    }
    __device__ __forceinline__ uint4 narrow() const {
        uint4 w;
        T* e = reinterpret_cast<T*>(&w);
#pragma unroll
        for (int i = 0; i < E; ++i) e[i] = from_float<T>(f[i]);
        return w;
    }
};

// Scale, zero and 1 / scale of the group whose smallest and largest element
// are mn, mx.  A group that is not finite keeps a zero that is not, and codes 0
// (inv and scale 0 for them), so that its bytes concern no other row.
__device__ __forceinline__ uint32_t int4_group_word(float mn, float mx, float& scale, float& inv, float& zero) {
    const __nv_bfloat16 z = __float2bfloat16_rd(mn + 0.f);   // (-0 becomes +0)
    zero = __bfloat162float(z);
    __nv_bfloat16 s = __float2bfloat16_ru(__fdiv_rn(__fsub_rn(mx, zero), 15.f));
    scale = __bfloat162float(s);
    if (scale > 0.f && scale < 1.17549435e-38f) {   // 2^-126: 1 / scale stays finite
        scale = 1.17549435e-38f;
        s = __float2bfloat16_rn(scale);
    }
    const uint32_t word = static_cast<uint32_t>(__bfloat16_as_ushort(s)) |
                          (static_cast<uint32_t>(__bfloat16_as_ushort(z)) << 16);
    if (!(scale < INFINITY)) scale = zero = 0.f;
    inv = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
    return word;
}

// The code of x in the low bits (four, of a finite group) of the result.  inv
// is 1 / scale rounded (0 where scale is 0): the product with it, corrected once
// by the exact remainder, is the rounded quotient (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990), so the
// code is the division's; the sum with 1.5 * 2^23 rounds it to a whole number.
// (The plain product is off next to ties, which 16-bit elements hit all the
// time; a division for each element costs twice this.)
__device__ __forceinline__ uint32_t code_bits(float x, float scale, float inv, float zero) {
    const float a = __fsub_rn(x, zero);
    const float q = __fmul_rn(a, inv);
    const float quotient = fmaf(fmaf(-q, scale, a), inv, q);
    return __float_as_uint(__fadd_rn(quotient, 12582912.f));
}

// Smaller and larger of two, not a number if one of them is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float m;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Writes lane `vec`'s vector v (dims vec * E ..) of a row into the tile of
// (block, head) at token t.  The D / E lanes of a row call it together
// (`mask`: every lane of the warp that does).
template <typename T, int D, Pool POOL>
__device__ __forceinline__ void write_row(const Vec<T>& v, uint8_t* pool, long long tile, int B, int t, int vec,
                                          bool value, float scale8, bool live, uint32_t mask) {
    constexpr int E = Vec<T>::E;
    if constexpr (POOL == Pool::kNative) {
        if (live)
            *reinterpret_cast<uint4*>(pool + tile * B * D * static_cast<int>(sizeof(T)) + (vec * B + t) * 16) =
                v.narrow();
    } else if constexpr (POOL == Pool::kE4m3) {
        if (!live) return;
        uint8_t* base = pool + tile * B * D;
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const int d = vec * E + i, e = d & 15;
            const uint32_t two = quantise2(v.f[i], v.f[i + 1], scale8);
            if (value) {
                base[d * B + v_row_byte(t, B)] = static_cast<uint8_t>(two);
                base[(d + 1) * B + v_row_byte(t, B)] = static_cast<uint8_t>(two >> 8);
            } else {
                *reinterpret_cast<uint16_t*>(base + ((d >> 4) * B + t) * 16 + 4 * ((e & 7) >> 1) + 2 * (e >> 3)) =
                    static_cast<uint16_t>(two);
            }
        }
    } else {
        constexpr int kLanes = kInt4Group / E;   // lanes that hold one group
        float mn = v.f[0], mx = v.f[0];
#pragma unroll
        for (int i = 1; i < E; ++i) {
            mn = min_nan(mn, v.f[i]);
            mx = max_nan(mx, v.f[i]);
        }
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) {
            mn = min_nan(mn, __shfl_xor_sync(mask, mn, off));
            mx = max_nan(mx, __shfl_xor_sync(mask, mx, off));
        }
        float scale, inv, zero;
        const uint32_t word = int4_group_word(mn, mx, scale, inv, zero);
        const bool finite = (word & 0x7f80u) != 0x7f80u;
        uint32_t own = 0;   // this lane's codes, four bits each
#pragma unroll
        for (int i = 0; i < E; ++i) {
            own |= (finite ? code_bits(v.f[i], scale, inv, zero) & 15u : 0u) << (4 * i);
        }
        // dims d and d + 8 meet in a byte: the lane 8 dims on holds the other nibble
        constexpr int kHop = 8 / E;
        const uint32_t other = __shfl_xor_sync(mask, own, kHop);
        const bool upper = (vec / kHop) & 1;
        const uint32_t lo = upper ? other : own, hi = upper ? own : other;
        if (!live) return;
        uint8_t* base = pool + tile * int4_tile_bytes(B, D);
        // the E bytes of the pair of lanes: the lower lane stores the first half
        const int d0 = (vec / (2 * kHop)) * 16 + (vec % kHop) * E;
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
            const int i = (upper ? E / 2 : 0) + j;
            base[int4_code_byte(value, B, D, t, d0 + i)] =
                static_cast<uint8_t>(((lo >> (4 * i)) & 15u) | (((hi >> (4 * i)) & 15u) << 4));
        }
        if (vec % kLanes == 0)
            *reinterpret_cast<uint32_t*>(base + B * D / 2 + (t * (D / kInt4Group) + vec / kLanes) * 4) = word;
    }
}

// ---- the 4-bit pools' write and read-back

struct RowsInt4Params {
    void* key;               // [T][Hkv][D] (the write reads, the read-back writes)
    void* value;
    uint8_t* k_cache;
    uint8_t* v_cache;
    const int64_t* slot_mapping;
    long long num_tokens;
    int num_kv_heads;
    int block_shift;         // log2 of the block size
    long long num_slots;
};

// One row, by the D / E lanes that hold it.
template <typename T, int D>
__device__ __forceinline__ void gather_row_int4(T* dst, const uint8_t* tile, int B, int t, int vec, bool value) {
    constexpr int E = Vec<T>::E;
    const uint32_t word = *reinterpret_cast<const uint32_t*>(
        tile + B * D / 2 + (t * (D / kInt4Group) + vec * E / kInt4Group) * 4);
    const float scale = __uint_as_float(word << 16), zero = __uint_as_float(word & 0xffff0000u);
    Vec<T> v;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int d = vec * E + e;
        const uint32_t byte = tile[int4_code_byte(value, B, D, t, d & ~8)];
        v.f[e] = fmaf(scale, static_cast<float>((d & 8) ? byte >> 4 : byte & 15u), zero);
    }
    *reinterpret_cast<uint4*>(dst + vec * E) = v.narrow();
}

// Row by row: a 16-byte vector of K and of V per thread.  For few tokens, whose
// slots lie anywhere (a decode step: latency).
template <typename T, int D, bool WRITE>
__global__ void __launch_bounds__(256) pa_rows_int4_kernel(const __grid_constant__ RowsInt4Params p) {
    wait_for_prior_work();
    constexpr int E = Vec<T>::E, V = D / E;
    // (this form takes few rows: 32-bit indices; the host sees to it)
    const int row = (blockIdx.x * 256 + threadIdx.x) / V, vec = threadIdx.x % V;
    const int i = row / p.num_kv_heads, h = row - i * p.num_kv_heads;
    const long long slot = i < p.num_tokens ? p.slot_mapping[i] : -1;
    if (slot >= p.num_slots) flag_error(4 /* PA_DEVERR_SLOT */);
    const bool live = slot >= 0 && slot < p.num_slots;
    const int B = 1 << p.block_shift;
    const long long block = live ? slot >> p.block_shift : 0;
    const int t = live ? static_cast<int>(slot) & (B - 1) : 0;
    const long long tile = block * p.num_kv_heads + h;
    if constexpr (WRITE) {
        Vec<T> k, v;
        const int at = live ? row * D + vec * E : 0;
        k.load(reinterpret_cast<const T*>(p.key) + at);
        v.load(reinterpret_cast<const T*>(p.value) + at);
        write_row<T, D, Pool::kInt4>(k, p.k_cache, tile, B, t, vec, false, 1.f, live, 0xffffffffu);
        write_row<T, D, Pool::kInt4>(v, p.v_cache, tile, B, t, vec, true, 1.f, live, 0xffffffffu);
    } else if (live) {
        const long long at = tile * int4_tile_bytes(B, D);
        gather_row_int4<T, D>(reinterpret_cast<T*>(p.key) + row * D, p.k_cache + at, B, t, vec, false);
        gather_row_int4<T, D>(reinterpret_cast<T*>(p.value) + row * D, p.v_cache + at, B, t, vec, true);
    }
}

// Transposes the 4 x 4 matrix that four neighbouring lanes (c = lane % 4) hold
// by rows: v[j] of lane c becomes v[c] of lane j.
__device__ __forceinline__ void transpose4(uint32_t (&v)[4], int c) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, (c & 1) ? v[j] : v[j + 1], 1);
        if (c & 1) v[j] = got; else v[j + 1] = got;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, (c & 2) ? v[j] : v[j + 2], 2);
        if (c & 2) v[j] = got; else v[j + 2] = got;
    }
}

// A group of G tokens (16; 8 with 8-token blocks) whose slots fill a group of
// the tile, one warp for one head, K or V: lane (r = lane / 4, m = lane % 4)
// takes tokens r (and r + 8) and, of every 64 dims, the m-th 16, whole rows of
// 16-byte vectors.  Its codes are its share of the four operand words of its
// 16 dims; a 4 x 4 transpose over the lanes of a row gives each lane the words
// it stores, one 16-byte vector of the tile.  A V word is the transpose of the
// 8 x 8 matrix of byte pairs that K words form (one movmatrix).  Row by row,
// every byte of the tile is a store of its own (8197 tokens: the write and the
// read-back took 53 us with that).
template <typename T, int D, int G>
__device__ __forceinline__ void write_group_int4(const T* src, long long row_stride, uint8_t* tile, int B, int t0,
                                                 int lane, bool value) {
    constexpr int NC = D / 64, NT = G / 8, E = Vec<T>::E;
    const int r = lane >> 2, m = lane & 3;
    uint8_t* codes = tile + (G == 16 ? (t0 >> 4) * NC * 512 : 0);
    uint32_t* groups = reinterpret_cast<uint32_t*>(tile + B * D / 2) + (t0 + r) * NC;
    // every load first: 16 dims of a row are 16 / E vectors
    uint4 raw[NC][NT][16 / E];
#pragma unroll
    for (int ch = 0; ch < NC; ++ch)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 16 / E; ++k)
                raw[ch][t][k] = *reinterpret_cast<const uint4*>(src + (r + 8 * t) * row_stride + ch * 64 + m * 16 + k * E);
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) {
        uint32_t byte[NT][8];   // dims d and d + 8 in the lowest byte
        uint32_t keep = 0u;     // the bytes of finite groups
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            Vec<T> x[16 / E];
#pragma unroll
            for (int k = 0; k < 16 / E; ++k) x[k].widen(raw[ch][t][k]);
            float mn = x[0].f[0], mx = mn;
#pragma unroll
            for (int d = 1; d < 16; ++d) {
                mn = min_nan(mn, x[d / E].f[d % E]);
                mx = max_nan(mx, x[d / E].f[d % E]);
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, off));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            }
            float scale, inv, zero;
            const uint32_t word = int4_group_word(mn, mx, scale, inv, zero);
            if ((word & 0x7f80u) != 0x7f80u) keep |= G == 16 ? 0x00ff00ffu << (8 * t) : 0xffffffffu;
            if (m == 0) groups[8 * t * NC + ch] = word;
#pragma unroll
            for (int d = 0; d < 8; ++d)
                byte[t][d] = code_bits(x[d / E].f[d % E], scale, inv, zero) +
                             (code_bits(x[(d + 8) / E].f[d % E], scale, inv, zero) << 4);
        }
        // the two dims 2j, 2j + 1: a byte each in both halves of the word, token r
        // in the lower, r + 8 in the upper
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (G == 16)
                w[j] = __byte_perm(__byte_perm(byte[0][2 * j], byte[NT - 1][2 * j], 0x0040),
                                   __byte_perm(byte[0][2 * j + 1], byte[NT - 1][2 * j + 1], 0x0040), 0x5410) & keep;
            else
                w[j] = __byte_perm(byte[0][2 * j], byte[0][2 * j + 1], 0x0400) & keep & 0x00ff00ffu;
        }
        transpose4(w, m);   // now the words of all four 16-dim tiles, dims 2m, 2m + 1
        if constexpr (G == 16) {
            if (value)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = movmatrix_trans(w[j]);
            *reinterpret_cast<uint4*>(codes + (ch * 32 + lane) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {   // 8-token blocks: a word holds two tiles, the second in the upper bytes
            uint32_t a = w[0] | (w[1] << 8), b = w[2] | (w[3] << 8);
            if (value) {
                a = movmatrix_trans(a);
                b = movmatrix_trans(b);
            }
            *reinterpret_cast<uint2*>(codes + (ch * 32 + lane) * 8) = make_uint2(a, b);
        }
    }
}

// The way back.
template <typename T, int D, int G>
__device__ __forceinline__ void gather_group_int4(T* dst, long long row_stride, const uint8_t* tile, int B, int t0,
                                                  int lane, bool value) {
    constexpr int NC = D / 64, NT = G / 8, E = Vec<T>::E;
    const int r = lane >> 2, m = lane & 3;
    const uint8_t* codes = tile + (G == 16 ? (t0 >> 4) * NC * 512 : 0);
    const uint32_t* groups = reinterpret_cast<const uint32_t*>(tile + B * D / 2) + (t0 + r) * NC;
    uint4 raw[NC];
    uint32_t word[NT][NC];
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) {
        if constexpr (G == 16) {
            raw[ch] = *reinterpret_cast<const uint4*>(codes + (ch * 32 + lane) * 16);
        } else {
            const uint2 a = *reinterpret_cast<const uint2*>(codes + (ch * 32 + lane) * 8);
            raw[ch].x = a.x;
            raw[ch].z = a.y;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) word[t][ch] = groups[8 * t * NC + ch];
    }
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) {
        uint32_t w[4] = {raw[ch].x, raw[ch].y, raw[ch].z, raw[ch].w};
        if constexpr (G == 16) {
            if (value)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = movmatrix_trans(w[j]);
        } else {
            if (value) {
                w[0] = movmatrix_trans(w[0]);
                w[2] = movmatrix_trans(w[2]);
            }
            w[1] = w[0] >> 8;
            w[3] = w[2] >> 8;
        }
        transpose4(w, m);   // this lane's 16 dims: dims 2j, 2j + 1 (and 8 on) in w[j]
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float scale = __uint_as_float(word[t][ch] << 16), zero = __uint_as_float(word[t][ch] & 0xffff0000u);
#pragma unroll
            for (int k = 0; k < 16 / E; ++k) {
                Vec<T> v;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int d = k * E + e;   // of 16
                    const uint32_t n = (w[d % 8 / 2] >> (8 * t + 16 * (d & 1) + 4 * (d >> 3))) & 15u;
                    v.f[e] = fmaf(scale, __uint_as_float(n | 0x4b000000u) - 8388608.f, zero);   // (2^23 + n)
                }
                *reinterpret_cast<uint4*>(dst + (r + 8 * t) * row_stride + ch * 64 + m * 16 + k * E) = v.narrow();
            }
        }
    }
}

// Many tokens: a warp takes the tokens [G w, G w + G) of one head's K or V, in
// groups where it can.  A token is part of a group if the G tokens from the one with
// offset 0 of its group in the block on (its leader) have consecutive slots;
// a warp writes the one group whose leader it holds (another cannot start
// within G tokens), and each of its tokens that is in no group by itself.  So a
// chunk that starts anywhere in a block goes by groups but for its ends.
template <typename T, int D, int G, bool WRITE>
__global__ void __launch_bounds__(128) pa_groups_int4_kernel(const __grid_constant__ RowsInt4Params p) {
    wait_for_prior_work();
    constexpr int E = Vec<T>::E, V = D / E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t unit = blockIdx.x * 4 + warp;   // (tokens, head, K or V), the last two first; below 2^32 (the host)
    const uint32_t set = unit / (2 * p.num_kv_heads);
    const long long i0 = static_cast<long long>(set) * G;
    const int hs = static_cast<int>(unit - set * 2 * p.num_kv_heads), h = hs >> 1;
    const bool value = hs & 1;
    if (i0 >= p.num_tokens) return;
    // slots of the tokens i0 - G .. i0 + 2 G - 1; lane k: tokens i0 - G + k and, from the 32nd on, i0 - G + 32 + k
    auto slot_at = [&](long long i) -> long long { return i >= 0 && i < p.num_tokens ? p.slot_mapping[i] : -1; };
    const long long a = slot_at(i0 - G + lane), b = 3 * G > 32 ? slot_at(i0 - G + 32 + lane) : -1;
    if (lane >= G && lane < 2 * G && a >= p.num_slots && hs == 0) flag_error(4 /* PA_DEVERR_SLOT */);
    // bit k: token i0 - G + k has a place in the pool and its follower the next one
    long long next = __shfl_down_sync(0xffffffffu, a, 1);
    const long long first_b = __shfl_sync(0xffffffffu, b, 0), next_b = __shfl_down_sync(0xffffffffu, b, 1);
    if (lane == 31) next = first_b;
    const uint64_t runs =
        __ballot_sync(0xffffffffu, a >= 0 && a < p.num_slots && next == a + 1 && next < p.num_slots) |
        (static_cast<uint64_t>(__ballot_sync(0xffffffffu, lane < 31 && b >= 0 && b < p.num_slots && next_b == b + 1 &&
                                                              next_b < p.num_slots))
         << 32);
    const uint64_t leads = __ballot_sync(0xffffffffu, a >= 0 && (a & (G - 1)) == 0);   // (of the first 32 tokens)
    constexpr uint64_t kRun = (1ull << (G - 1)) - 1;
    // bit k: a group starts at token i0 - G + k, k < 2 G
    uint64_t groups = leads;
#pragma unroll
    for (int j = 0; j < G - 1; ++j) groups &= runs >> j;
    static_assert(2 * G <= 32 && kRun != 0, "leaders within the first 32 tokens");
    const int B = 1 << p.block_shift;
    const long long stride = static_cast<long long>(p.num_kv_heads) * D;
    T* rows = reinterpret_cast<T*>(value ? p.value : p.key) + h * D;
    uint8_t* pool = value ? p.v_cache : p.k_cache;
    const uint32_t mine = static_cast<uint32_t>(groups >> G) & ((1u << G) - 1u);
    if (mine != 0u) {
        const int k = __ffs(mine) - 1;
        const long long slot = __shfl_sync(0xffffffffu, a, G + k);
        const long long tile = ((slot >> p.block_shift) * p.num_kv_heads + h) * int4_tile_bytes(B, D);
        const int t0 = static_cast<int>(slot) & (B - 1);
        if constexpr (WRITE)
            write_group_int4<T, D, G>(rows + (i0 + k) * stride, stride, pool + tile, B, t0, lane, value);
        else
            gather_group_int4<T, D, G>(rows + (i0 + k) * stride, stride, pool + tile, B, t0, lane, value);
    }
    // tokens of this warp in no group: no group starts at one of the G tokens up to it
    uint32_t alone = 0u;
#pragma unroll
    for (int k = 0; k < G; ++k)
        if (((groups >> (k + 1)) & ((1ull << G) - 1)) == 0) alone |= 1u << k;
    alone &= static_cast<uint32_t>(__ballot_sync(0xffffffffu, a >= 0 && a < p.num_slots) >> G);
    alone &= (1u << G) - 1u;
    constexpr int kRows = 32 / V;   // rows the warp takes at once
    while (alone != 0u) {
        uint32_t rest = alone;
        int k = -1;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {   // row j of the warp: the j-th lowest token
            const int bit = rest != 0u ? __ffs(rest) - 1 : -1;
            if (lane / V == j) k = bit;
            rest &= rest - 1u;   // (0 stays 0)
        }
        alone = rest;
        const long long slot = __shfl_sync(0xffffffffu, a, G + (k < 0 ? 0 : k));
        const bool live = k >= 0;
        const long long tile = (live ? slot >> p.block_shift : 0) * p.num_kv_heads + h;
        const int t = live ? static_cast<int>(slot) & (B - 1) : 0, vec = lane % V;
        T* row = rows + (i0 + (live ? k : 0)) * stride;
        if constexpr (WRITE) {
            Vec<T> x;
            x.load(row + vec * E);
            write_row<T, D, Pool::kInt4>(x, pool, tile, B, t, vec, value, 1.f, live, 0xffffffffu);
        } else if (live) {
            gather_row_int4<T, D>(row, pool + tile * int4_tile_bytes(B, D), B, t, vec, value);
        }
    }
}

}  // namespace pa
