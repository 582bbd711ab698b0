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

// Scale and zero of the group whose smallest and largest element are mn, mx.
__device__ __forceinline__ uint32_t int4_group_word(float mn, float mx, float& scale, float& zero) {
    const __nv_bfloat16 z = __float2bfloat16_rd(mn + 0.f);   // (-0 becomes +0)
    zero = __bfloat162float(z);
    __nv_bfloat16 s = __float2bfloat16_ru(__fdiv_rn(__fsub_rn(mx, zero), 15.f));
    scale = __bfloat162float(s);
    if (scale > 0.f && scale < 1.17549435e-38f) {   // 2^-126: the quotients below stay finite
        scale = 1.17549435e-38f;
        s = __float2bfloat16_rn(scale);
    }
    return static_cast<uint32_t>(__bfloat16_as_ushort(s)) | (static_cast<uint32_t>(__bfloat16_as_ushort(z)) << 16);
}

// The code of x, by the definition (0 for what is not a number).
__device__ __forceinline__ float whole_code(float x, float scale, float zero) {
    const float n = scale > 0.f ? rintf(__fdiv_rn(__fsub_rn(x, zero), scale)) : 0.f;
    return fminf(fmaxf(n, 0.f), 15.f);
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
            mn = fminf(mn, v.f[i]);
            mx = fmaxf(mx, v.f[i]);
        }
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) {
            mn = fminf(mn, __shfl_xor_sync(mask, mn, off));
            mx = fmaxf(mx, __shfl_xor_sync(mask, mx, off));
        }
        float scale, zero;
        const uint32_t word = int4_group_word(mn, mx, scale, zero);
        uint32_t own = 0;   // this lane's codes, four bits each
#pragma unroll
        for (int i = 0; i < E; ++i) {
            own |= static_cast<uint32_t>(whole_code(v.f[i], scale, zero)) << (4 * i);
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
    int block_size;
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
    const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long row = idx / V;
    const int vec = static_cast<int>(idx % V);
    const long long i = row / p.num_kv_heads;
    const int h = static_cast<int>(row - i * p.num_kv_heads);
    const long long slot = i < p.num_tokens ? p.slot_mapping[i] : -1;
    if (slot >= p.num_slots) flag_error(4 /* PA_DEVERR_SLOT */);
    const bool live = slot >= 0 && slot < p.num_slots;
    const long long block = live ? slot / p.block_size : 0;
    const int t = live ? static_cast<int>(slot - block * p.block_size) : 0;
    const long long tile = block * p.num_kv_heads + h;
    if constexpr (WRITE) {
        Vec<T> k, v;
        const long long at = live ? row * D + vec * E : 0;
        k.load(reinterpret_cast<const T*>(p.key) + at);
        v.load(reinterpret_cast<const T*>(p.value) + at);
        write_row<T, D, Pool::kInt4>(k, p.k_cache, tile, p.block_size, t, vec, false, 1.f, live, 0xffffffffu);
        write_row<T, D, Pool::kInt4>(v, p.v_cache, tile, p.block_size, t, vec, true, 1.f, live, 0xffffffffu);
    } else if (live) {
        const long long at = tile * int4_tile_bytes(p.block_size, D);
        gather_row_int4<T, D>(reinterpret_cast<T*>(p.key) + row * D, p.k_cache + at, p.block_size, t, vec, false);
        gather_row_int4<T, D>(reinterpret_cast<T*>(p.value) + row * D, p.v_cache + at, p.block_size, t, vec, true);
    }
}

// Two neighbouring elements.
template <typename T>
__device__ __forceinline__ float2 load2(const T* p) {
    if constexpr (sizeof(T) == 4) {
        return *reinterpret_cast<const float2*>(p);
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
        const T* e = reinterpret_cast<const T*>(&w);
        return make_float2(to_float<T>(e[0]), to_float<T>(e[1]));
    }
}
template <typename T>
__device__ __forceinline__ void store2(T* p, float a, float b) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float2*>(p) = make_float2(a, b);
    } else {
        uint32_t w;
        T* e = reinterpret_cast<T*>(&w);
        e[0] = from_float<T>(a);
        e[1] = from_float<T>(b);
        *reinterpret_cast<uint32_t*>(p) = w;
    }
}

// A group of G tokens (16; 8 with 8-token blocks) whose slots fill a group of
// the tile, one warp for one head: lane (r = lane / 4, c = lane % 4) takes
// tokens r (and r + 8) and, of every 16 dims, 2c, 2c + 1, 2c + 8, 2c + 9, which
// is its operand word of K; a V word is the transpose of the 8 x 8 matrix of
// byte pairs that such words form (one movmatrix).  So a lane reads and writes
// whole words of 16-byte vectors of the tile, where the row by row form stores
// every byte by itself (8197 tokens: the write and read-back 53 us with it).
//
// The quotient is taken by the reciprocal, whose product is off by at most 3e-6
// (15 * 1.5 * 2^-23); it rounds to the same whole number as the division's
// unless that lies within 1e-5 of a half, and then the division is done.
template <typename T, int D, int G>
__device__ __forceinline__ void write_group_int4(const T* src, long long row_stride, uint8_t* tile, int B, int t0,
                                                 int lane, bool value) {
    constexpr int NC = D / 64, NT = G / 8, W = G == 16 ? 4 : 2;
    const int r = lane >> 2, c = lane & 3;
    uint8_t* codes = tile + (G == 16 ? (t0 >> 4) * NC * 512 : 0);
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) {
        float2 pair[NT][4][2];   // token, 16-dim tile, dims 2c / 2c + 8
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    pair[t][m][u] = load2<T>(src + (r + 8 * t) * row_stride + ch * 64 + m * 16 + u * 8 + 2 * c);
        float code[NT][4][2][2];   // token, tile, odd dim, upper: whole numbers
        uint32_t words[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float mn = pair[t][0][0].x, mx = mn;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    mn = fminf(mn, fminf(pair[t][m][u].x, pair[t][m][u].y));
                    mx = fmaxf(mx, fmaxf(pair[t][m][u].x, pair[t][m][u].y));
                }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            }
            float scale, zero;
            words[t] = int4_group_word(mn, mx, scale, zero);
            const float inv = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
            bool near_half = false;   // (or not a number: what is not finite must not reach another token's bytes)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        const float q = __fmul_rn(__fsub_rn(odd ? pair[t][m][u].y : pair[t][m][u].x, zero), inv);
                        const float n = __fsub_rn(__fadd_rn(q, 12582912.f), 12582912.f);   // 1.5 2^23: to the nearest whole
                        near_half |= !(fabsf(q - n) <= 0.49999f);
                        code[t][m][odd][u] = n;
                    }
            if (near_half) {
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int odd = 0; odd < 2; ++odd)
                            code[t][m][odd][u] = whole_code(odd ? pair[t][m][u].y : pair[t][m][u].x, scale, zero);
            }
        }
        // words: two bytes (token r and r + 8; 8-token blocks: tiles 2j and 2j + 1)
        // of each of the two dims, summed as whole numbers below 2^16
        uint32_t w[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            uint32_t half[2];
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
                const float(&lo)[2] = G == 16 ? code[0][j % 4][odd] : code[0][2 * (j % 2)][odd];
                const float(&hi)[2] = G == 16 ? code[NT - 1][j % 4][odd] : code[0][2 * (j % 2) + 1][odd];
                const float sum = fmaf(256.f, fmaf(16.f, hi[1], hi[0]), fmaf(16.f, lo[1], lo[0]));
                half[odd] = __float_as_uint(sum + 8388608.f);
            }
            w[j] = __byte_perm(half[0], half[1], 0x5410);
            if (value) w[j] = movmatrix_trans(w[j]);
        }
        if constexpr (W == 4)
            *reinterpret_cast<uint4*>(codes + (ch * 32 + lane) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2*>(codes + (ch * 32 + lane) * 8) = make_uint2(w[0], w[1]);
        if (c == 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                *reinterpret_cast<uint32_t*>(tile + B * D / 2 + ((t0 + r + 8 * t) * NC + ch) * 4) = words[t];
        }
    }
}

template <typename T, int D, int G>
__device__ __forceinline__ void gather_group_int4(T* dst, long long row_stride, const uint8_t* tile, int B, int t0,
                                                  int lane, bool value) {
    constexpr int NC = D / 64, NT = G / 8, W = G == 16 ? 4 : 2;
    const int r = lane >> 2, c = lane & 3;
    const uint8_t* codes = tile + (G == 16 ? (t0 >> 4) * NC * 512 : 0);
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) {
        uint32_t w[W];
        if constexpr (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(codes + (ch * 32 + lane) * 16);
            w[0] = x.x;
            w[1] = x.y;
            w[2] = x.z;
            w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(codes + (ch * 32 + lane) * 8);
            w[0] = x.x;
            w[1] = x.y;
        }
        float scale[NT], zero[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t g =
                *reinterpret_cast<const uint32_t*>(tile + B * D / 2 + ((t0 + r + 8 * t) * NC + ch) * 4);
            scale[t] = __uint_as_float(g << 16);
            zero[t] = __uint_as_float(g & 0xffff0000u);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (value) w[j] = movmatrix_trans(w[j]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {   // bytes b and b + 2: dims 2c and 2c + 1
                const int t = G == 16 ? b : 0, m = G == 16 ? j % 4 : 2 * (j % 2) + b;
                T* row = dst + (r + 8 * t) * row_stride + ch * 64 + m * 16 + 2 * c;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float f[2];
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        const uint32_t n = (w[j] >> (8 * b + 16 * odd + 4 * u)) & 15u;
                        f[odd] = fmaf(scale[t], __uint_as_float(n | 0x4b000000u) - 8388608.f, zero[t]);
                    }
                    store2<T>(row + 8 * u, f[0], f[1]);
                }
            }
        }
    }
}

// Many tokens: a warp takes the tokens [G w, G w + G) of one head, in groups
// where it can.  A token is part of a group if the G tokens from the one with
// offset 0 of its group in the block on (its leader) have consecutive slots;
// a warp writes the one group whose leader it holds (another cannot start
// within G tokens), and each of its tokens that is in no group by itself.  So a
// chunk that starts anywhere in a block goes by groups but for its ends.
template <typename T, int D, int G, bool WRITE>
__global__ void __launch_bounds__(128) pa_groups_int4_kernel(const __grid_constant__ RowsInt4Params p) {
    wait_for_prior_work();
    constexpr int E = Vec<T>::E, V = D / E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * 4 + warp;   // (tokens, head), heads first
    const long long i0 = unit / p.num_kv_heads * G;
    const int h = static_cast<int>(unit % p.num_kv_heads);
    if (i0 >= p.num_tokens) return;
    // slots of the tokens i0 - G .. i0 + 2 G - 1; lane k: tokens i0 - G + k and, from the 32nd on, i0 - G + 32 + k
    auto slot_at = [&](long long i) -> long long { return i >= 0 && i < p.num_tokens ? p.slot_mapping[i] : -1; };
    const long long a = slot_at(i0 - G + lane), b = 3 * G > 32 ? slot_at(i0 - G + 32 + lane) : -1;
    if (lane >= G && lane < 2 * G && a >= p.num_slots && h == 0) flag_error(4 /* PA_DEVERR_SLOT */);
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
    const int B = p.block_size;
    const long long stride = static_cast<long long>(p.num_kv_heads) * D;
    T* key = reinterpret_cast<T*>(p.key) + h * D;
    T* value = reinterpret_cast<T*>(p.value) + h * D;
    const uint32_t mine = static_cast<uint32_t>(groups >> G) & ((1u << G) - 1u);
    if (mine != 0u) {
        const int k = __ffs(mine) - 1;
        const long long slot = __shfl_sync(0xffffffffu, a, G + k);
        const long long block = slot / B, tile = (block * p.num_kv_heads + h) * int4_tile_bytes(B, D);
        const int t0 = static_cast<int>(slot - block * B);
        const long long at = (i0 + k) * stride;
        if constexpr (WRITE) {
            write_group_int4<T, D, G>(key + at, stride, p.k_cache + tile, B, t0, lane, false);
            write_group_int4<T, D, G>(value + at, stride, p.v_cache + tile, B, t0, lane, true);
        } else {
            gather_group_int4<T, D, G>(key + at, stride, p.k_cache + tile, B, t0, lane, false);
            gather_group_int4<T, D, G>(value + at, stride, p.v_cache + tile, B, t0, lane, true);
        }
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
        const long long block = live ? slot / B : 0, tile = block * p.num_kv_heads + h;
        const int t = live ? static_cast<int>(slot - block * B) : 0, vec = lane % V;
        const long long at = (i0 + (live ? k : 0)) * stride;
        if constexpr (WRITE) {
            Vec<T> x, y;
            x.load(key + at + vec * E);
            y.load(value + at + vec * E);
            write_row<T, D, Pool::kInt4>(x, p.k_cache, tile, B, t, vec, false, 1.f, live, 0xffffffffu);
            write_row<T, D, Pool::kInt4>(y, p.v_cache, tile, B, t, vec, true, 1.f, live, 0xffffffffu);
        } else if (live) {
            gather_row_int4<T, D>(key + at, p.k_cache + tile * int4_tile_bytes(B, D), B, t, vec, false);
            gather_row_int4<T, D>(value + at, p.v_cache + tile * int4_tile_bytes(B, D), B, t, vec, true);
        }
    }
}

}  // namespace pa
