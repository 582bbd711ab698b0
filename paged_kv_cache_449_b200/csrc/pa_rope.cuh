// Rotary positions, head norms and the cache write in one pass: the step
// between the projections and the attention.  For every token i at position
// pos_i and every head, x the head's row of q or k:
//     x <- x / sqrt(mean(x^2) + eps) * weight          (optional, fp32)
//     (x_a, x_b) <- m (x_a cos - x_b sin, x_b cos + x_a sin),  angle = pos_i * inv_freq[j]
// over the pairs j < R / 2 of the first R dims: (j, j + R/2) in the half
// layout, (2j, 2j + 1) interleaved; dims from R on pass through.  q goes to
// q_out, k and v into the pool at the token's slot (slot < 0: q only).  Each
// element is rounded once.
//
// The angle is exact: the product is formed in fp64 in units of a turn and the
// whole turns dropped before fp32 sine and cosine (fp32 products of far
// positions are off by whole tenths of a radian).  It costs a few fp64
// operations per token and frequency, shared by every head of the token.
//
// Bound by memory: 2 (Hq + 2 Hkv) D e bytes a token.
#pragma once

#include "pa_rows.cuh"

namespace pa {

struct RopeParams {
    void* q_out;              // [T][Hq][D]
    const void* q;            // [T] rows q_stride elements apart, each [Hq][D]
    const void* key;          // [T] rows k_stride apart, [Hkv][D]
    const void* value;
    uint8_t* k_cache;
    uint8_t* v_cache;
    const int64_t* positions;     // [T]
    const int64_t* slot_mapping;  // [T]
    const float* inv_freq;        // [R / 2]
    const void* q_weight;         // [D] or null (no norm)
    const void* k_weight;
    const float* k_scale;         // 8-bit pools: [Hkv]
    const float* v_scale;
    long long q_stride, k_stride, v_stride;
    float rope_scale;             // m
    float eps;
    int num_q_heads;
    int num_kv_heads;
    int rotary_dim;               // R
    int block_shift;              // log2 of the block size
    long long num_slots;
};

#ifndef PA_ROPE_ROWS
#define PA_ROPE_ROWS 3
#endif
#ifndef PA_ROPE_CTAS
#define PA_ROPE_CTAS 4
#endif
constexpr int kRopeRows = PA_ROPE_ROWS;
constexpr int kRopeThreads = 256;   // at most

// One CTA per token, of 64 threads (many tokens) to 256 (few); a group of D / E lanes takes one head's row at a time,
// kRopeRows rows in flight: their loads are asked for first, then the token's
// sines and cosines computed while they come.
template <typename T, int D, Pool POOL, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, POOL == Pool::kNative ? PA_ROPE_CTAS : 3) pa_rope_cache_kernel(const __grid_constant__ RopeParams p) {
    wait_for_prior_work();
    constexpr int E = Vec<T>::E, V = D / E;
    const int step = blockDim.x / V;         // rows the CTA takes at once
    __shared__ float2 turn[D / 2];            // m cos, m sin
    const long long i = blockIdx.x;
    const long long slot = p.slot_mapping[i];
    const int vec = threadIdx.x % V, lane = threadIdx.x & 31;
    const int rows = p.num_q_heads + 2 * p.num_kv_heads, v_row = p.num_q_heads + p.num_kv_heads;
    const int half = p.rotary_dim / 2;
    const bool live = slot >= 0 && slot < p.num_slots;

    uint4 raw[kRopeRows];
    auto load = [&](int r0) {
#pragma unroll
        for (int k = 0; k < kRopeRows; ++k) {
            const int row = r0 + k * step;
            const T* src = reinterpret_cast<const T*>(p.q) + i * p.q_stride + row * D;
            if (row >= p.num_q_heads) src = reinterpret_cast<const T*>(p.key) + i * p.k_stride + (row - p.num_q_heads) * D;
            if (row >= v_row) src = reinterpret_cast<const T*>(p.value) + i * p.v_stride + (row - v_row) * D;
            raw[k] = row < rows ? *reinterpret_cast<const uint4*>(src + vec * E) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    const int first = threadIdx.x / V;
    load(first);
    for (int j = threadIdx.x; j < half; j += blockDim.x) {
        const double turns =
            static_cast<double>(p.positions[i]) * (static_cast<double>(p.inv_freq[j]) * 0.15915494309189533577);
        const float part = static_cast<float>(turns - rint(turns));   // of a turn, [-1/2, 1/2]
        float s, c;
        sincospif(2.f * part, &s, &c);
        turn[j] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
    if (slot >= p.num_slots && threadIdx.x == 0) flag_error(4 /* PA_DEVERR_SLOT */);
    const int block_size = 1 << p.block_shift;
    const long long block = live ? slot >> p.block_shift : 0;
    const int t = live ? static_cast<int>(slot) & (block_size - 1) : 0;
    __syncthreads();
    // This thread's dims are the same in every row, and so are its angles.
    // Half layout: x' = x cos + y sin', y the pair's other element, which lies
    // half / E lanes away, sin' = -sin in the pair's first half.
    const int hop = half / E;
    const bool low = vec < hop, turned = INTERLEAVED ? vec * E < p.rotary_dim : vec < 2 * hop;
    const int from = turned ? lane + (low ? hop : -hop) : lane;
    constexpr int kPairs = INTERLEAVED ? E / 2 : E;
    float cs[kPairs], sn[kPairs];
    if (turned) {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            const float2 a = turn[INTERLEAVED ? vec * (E / 2) + e : (low ? vec : vec - hop) * E + e];
            cs[e] = a.x;
            sn[e] = !INTERLEAVED && low ? -a.y : a.y;
        }
    }

    // every lane of a warp takes the same number of turns: the shuffles stay whole
    for (int r0 = first; r0 - first < rows; r0 += kRopeRows * step) {
#pragma unroll
        for (int k = 0; k < kRopeRows; ++k) {
            const int row = r0 + k * step;
            if (row - first >= rows) break;   // (uniform)
            const bool in = row < rows, is_q = row < p.num_q_heads, is_v = row >= v_row;
            const int h = is_q ? row : (is_v ? row - v_row : row - p.num_q_heads);
            const bool write = in && !is_q && live;
            const long long tile = write ? block * p.num_kv_heads + h : 0;
            if (POOL == Pool::kNative && __all_sync(0xffffffffu, is_v)) {   // a warp of V rows: copied as they are
                if (write)
                    *reinterpret_cast<uint4*>(p.v_cache + tile * block_size * D * static_cast<int>(sizeof(T)) +
                                              (vec * block_size + t) * 16) = raw[k];
                continue;
            }
            Vec<T> x;
            x.widen(raw[k]);
            if constexpr (NORM) {
                const T* w = reinterpret_cast<const T*>(is_q ? p.q_weight : p.k_weight);
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) sum = fmaf(x.f[e], x.f[e], sum);
#pragma unroll
                for (int off = 1; off < V; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (!is_v && w != nullptr) {
                    const float inv = rsqrtf(sum * (1.f / D) + p.eps);
                    Vec<T> g;
                    g.load(w + vec * E);
#pragma unroll
                    for (int e = 0; e < E; ++e) x.f[e] = x.f[e] * inv * g.f[e];
                }
            }
            if constexpr (INTERLEAVED) {
                if (turned && !is_v) {
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float a = x.f[e], b = x.f[e + 1];
                        x.f[e] = a * cs[e / 2] - b * sn[e / 2];
                        x.f[e + 1] = b * cs[e / 2] + a * sn[e / 2];
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float y = __shfl_sync(0xffffffffu, x.f[e], from);
                    if (turned && !is_v) x.f[e] = x.f[e] * cs[e] + y * sn[e];
                }
            }
            if (is_q && in)
                *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.q_out) + (i * p.num_q_heads + h) * D + vec * E) = x.narrow();
            if (__all_sync(0xffffffffu, is_q)) continue;
            float scale8 = 1.f;
            if constexpr (POOL == Pool::kE4m3) scale8 = write ? (is_v ? p.v_scale : p.k_scale)[h] : 1.f;
            if constexpr (POOL != Pool::kNative) {   // (what a quantised pool holds is the rounded row's code)
#pragma unroll
                for (int e = 0; e < E; ++e) x.f[e] = to_float<T>(from_float<T>(x.f[e]));
            }
            write_row<T, D, POOL>(x, is_v ? p.v_cache : p.k_cache, tile, block_size, t, vec, is_v, scale8, write,
                                  0xffffffffu);
        }
        if (r0 - first + kRopeRows * step < rows) load(r0 + kRopeRows * step);
    }
}

}  // namespace pa
