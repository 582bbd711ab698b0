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
            const float x = scale > 0.f ? rintf(__fdiv_rn(__fsub_rn(v.f[i], zero), scale)) : 0.f;
            own |= static_cast<uint32_t>(fminf(fmaxf(x, 0.f), 15.f)) << (4 * i);
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

// ---- the 4-bit pools' write and read-back: one 16-byte vector of K and one of V per thread

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

template <typename T, int D>
__global__ void __launch_bounds__(256) pa_reshape_int4_kernel(const __grid_constant__ RowsInt4Params p) {
    wait_for_prior_work();
    constexpr int E = Vec<T>::E, V = D / E;
    const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long row = idx / V;
    const int vec = static_cast<int>(idx % V);
    const long long i = row / p.num_kv_heads;
    const int h = static_cast<int>(row - i * p.num_kv_heads);
    const bool in = i < p.num_tokens;
    const long long slot = in ? p.slot_mapping[i] : -1;
    if (slot >= p.num_slots) flag_error(4 /* PA_DEVERR_SLOT */);
    const bool live = slot >= 0 && slot < p.num_slots;
    Vec<T> k, v;
    const long long at = live ? row * D + vec * E : 0;
    k.load(reinterpret_cast<const T*>(p.key) + at);
    v.load(reinterpret_cast<const T*>(p.value) + at);
    const long long block = live ? slot / p.block_size : 0;
    const int t = live ? static_cast<int>(slot - block * p.block_size) : 0;
    const long long tile = block * p.num_kv_heads + h;
    write_row<T, D, Pool::kInt4>(k, p.k_cache, tile, p.block_size, t, vec, false, 1.f, live, 0xffffffffu);
    write_row<T, D, Pool::kInt4>(v, p.v_cache, tile, p.block_size, t, vec, true, 1.f, live, 0xffffffffu);
}

// The values at slots, rounded once to T; rows of negative slots keep what they held.
template <typename T, int D>
__global__ void __launch_bounds__(256) pa_gather_int4_kernel(const __grid_constant__ RowsInt4Params p) {
    wait_for_prior_work();
    constexpr int E = Vec<T>::E, V = D / E;
    const long long idx = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long row = idx / V;
    const int vec = static_cast<int>(idx % V);
    const long long i = row / p.num_kv_heads;
    const int h = static_cast<int>(row - i * p.num_kv_heads);
    if (i >= p.num_tokens) return;
    const long long slot = p.slot_mapping[i];
    if (slot < 0) return;
    if (slot >= p.num_slots) {
        flag_error(4 /* PA_DEVERR_SLOT */);
        return;
    }
    const int B = p.block_size;
    const long long block = slot / B;
    const int t = static_cast<int>(slot - block * B);
    const long long tile = (block * p.num_kv_heads + h) * int4_tile_bytes(B, D);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const uint8_t* base = (side ? p.v_cache : p.k_cache) + tile;
        const uint32_t word = *reinterpret_cast<const uint32_t*>(
            base + B * D / 2 + (t * (D / kInt4Group) + vec * E / kInt4Group) * 4);
        const float scale = __uint_as_float(word << 16), zero = __uint_as_float(word & 0xffff0000u);
        Vec<T> v;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = vec * E + e;
            const uint32_t byte = base[int4_code_byte(side, B, D, t, d & ~8)];
            v.f[e] = fmaf(scale, static_cast<float>((d & 8) ? byte >> 4 : byte & 15u), zero);
        }
        *reinterpret_cast<uint4*>(reinterpret_cast<T*>(side ? p.value : p.key) + row * D + vec * E) = v.narrow();
    }
}

}  // namespace pa
