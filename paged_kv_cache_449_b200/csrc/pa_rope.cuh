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

constexpr int kRopeRows = 3;         // rows a thread has in flight (2: 37.9 us, 4: 40.2, 3: 37.4 at 6166 tokens)
constexpr int kRopeThreads = 256;   // at most

// One CTA per token, of 64 threads (many tokens) to 256 (few); a group of D / E
// lanes takes one head's row at a time, kRopeRows rows in flight.  The rows of
// q, k and v are three loops, so that what differs between them (the source,
// the norm's weights, where a row goes) is set up once; the first rows are asked
// for before the token's sines and cosines are computed.
template <typename T, int D, Pool POOL, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, POOL == Pool::kNative ? 4 : 3) pa_rope_cache_kernel(const __grid_constant__ RopeParams p) {
    wait_for_prior_work();
    constexpr int E = Vec<T>::E, V = D / E;
    __shared__ float2 turn[D / 2];            // m cos, m sin
    const long long i = blockIdx.x;
    const int vec = threadIdx.x % V, lane = threadIdx.x & 31, first = threadIdx.x / V;
    const int step = blockDim.x / V;          // rows the CTA takes at once
    const int half = p.rotary_dim / 2;
    const T* qsrc = reinterpret_cast<const T*>(p.q) + i * p.q_stride + vec * E;
    const T* ksrc = reinterpret_cast<const T*>(p.key) + i * p.k_stride + vec * E;
    const T* vsrc = reinterpret_cast<const T*>(p.value) + i * p.v_stride + vec * E;
    uint4 raw[kRopeRows];
    auto load = [&](const T* src, int heads, int base) {   // rows base + first, + step, ..
#pragma unroll
        for (int k = 0; k < kRopeRows; ++k) {
            const int h = base + k * step + first;
            raw[k] = h < heads ? *reinterpret_cast<const uint4*>(src + h * D) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load(qsrc, p.num_q_heads, 0);
    const long long slot = p.slot_mapping[i];
    for (int j = threadIdx.x; j < half; j += blockDim.x) {
        const double turns =
            static_cast<double>(p.positions[i]) * (static_cast<double>(p.inv_freq[j]) * 0.15915494309189533577);
        const float part = static_cast<float>(turns - rint(turns));   // of a turn, [-1/2, 1/2]
        float s, c;
        sincospif(2.f * part, &s, &c);
        turn[j] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
    const bool live = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && threadIdx.x == 0) flag_error(4 /* PA_DEVERR_SLOT */);
    const int block_size = 1 << p.block_shift;
    const int t = live ? static_cast<int>(slot) & (block_size - 1) : 0;
    const long long tile0 = (live ? slot >> p.block_shift : 0) * p.num_kv_heads;
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
    // norm and rotation of one row (every lane of the warp takes part)
    auto turn_row = [&](Vec<T>& x, const Vec<T>& g, bool norm) {
        if (NORM && norm) {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) sum = fmaf(x.f[e], x.f[e], sum);
#pragma unroll
            for (int off = 1; off < V; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            const float inv = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
            for (int e = 0; e < E; ++e) x.f[e] = x.f[e] * inv * g.f[e];
        }
        if constexpr (INTERLEAVED) {
            if (turned) {
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
                if (turned) x.f[e] = x.f[e] * cs[e] + y * sn[e];
            }
        }
    };
    // a row of k or v into its tile
    auto keep = [&](Vec<T>& x, uint8_t* pool, const float* scale, int h, bool in, bool value) {
        const bool write = in && live;
        float scale8 = 1.f;
        if constexpr (POOL == Pool::kE4m3) scale8 = write ? scale[h] : 1.f;
        if constexpr (POOL != Pool::kNative) {   // (what a quantised pool holds is the rounded row's code)
#pragma unroll
            for (int e = 0; e < E; ++e) x.f[e] = to_float<T>(from_float<T>(x.f[e]));
        }
        write_row<T, D, POOL>(x, pool, write ? tile0 + h : 0, block_size, t, vec, value, scale8, write, 0xffffffffu);
    };
    Vec<T> g;
    if (NORM && p.q_weight != nullptr) g.load(reinterpret_cast<const T*>(p.q_weight) + vec * E);
    T* q_out = reinterpret_cast<T*>(p.q_out) + i * p.num_q_heads * D + vec * E;
    for (int base = 0; base < p.num_q_heads; base += kRopeRows * step) {
        if (base > 0) load(qsrc, p.num_q_heads, base);
#pragma unroll
        for (int k = 0; k < kRopeRows; ++k) {
            if (base + k * step >= p.num_q_heads) break;   // (uniform)
            const int h = base + k * step + first;
            Vec<T> x;
            x.widen(raw[k]);
            turn_row(x, g, p.q_weight != nullptr);
            if (h < p.num_q_heads) *reinterpret_cast<uint4*>(q_out + h * D) = x.narrow();
        }
    }
    if (!live) return;   // (the whole block: a token without a place keeps its q only)
    if (NORM && p.k_weight != nullptr) g.load(reinterpret_cast<const T*>(p.k_weight) + vec * E);
    for (int base = 0; base < p.num_kv_heads; base += kRopeRows * step) {
        load(ksrc, p.num_kv_heads, base);
#pragma unroll
        for (int k = 0; k < kRopeRows; ++k) {
            if (base + k * step >= p.num_kv_heads) break;
            const int h = base + k * step + first;
            Vec<T> x;
            x.widen(raw[k]);
            turn_row(x, g, p.k_weight != nullptr);
            keep(x, p.k_cache, p.k_scale, h, h < p.num_kv_heads, false);
        }
    }
    for (int base = 0; base < p.num_kv_heads; base += kRopeRows * step) {
        load(vsrc, p.num_kv_heads, base);
#pragma unroll
        for (int k = 0; k < kRopeRows; ++k) {
            if (base + k * step >= p.num_kv_heads) break;
            const int h = base + k * step + first;
            if constexpr (POOL == Pool::kNative) {   // as it is
                if (h < p.num_kv_heads)
                    *reinterpret_cast<uint4*>(p.v_cache + (tile0 + h) * block_size * D * static_cast<int>(sizeof(T)) +
                                              (vec * block_size + t) * 16) = raw[k];
            } else {
                Vec<T> x;
                x.widen(raw[k]);
                keep(x, p.v_cache, p.v_scale, h, h < p.num_kv_heads, true);
            }
        }
    }
}

}  // namespace pa
