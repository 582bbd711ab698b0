// Host side of the C ABI declared in include/pa/ops.h: rotary positions with
// the cache write, 4-bit pools, sliding windows.
//
// A translation unit of its own (the library's kernels compile side by side),
// and so with a device error word of its own, which pa_get_device_error reads
// and clears with the other (pa_ops_take_error).
#include "pa_host.cuh"

#include "pa/ops.h"
#include "pa_decode_int4.cuh"
#include "pa_rope.cuh"
#include "pa_rows.cuh"

namespace {

// The most blocks of `unit` tokens that hold a visible token of one sequence.
long long visible_units(long long cap, long long window, long long sinks, int unit) {
    const long long all = (cap + unit - 1) / unit;
    if (window <= 0) return all;
    const long long some = (window + unit - 2) / unit + 1 + (sinks + unit - 1) / unit;
    return std::min(all, some);
}

// Partitions of `partition_size` tokens (0: one) that the visible units need.
long long window_partitions(long long units, int unit, int partition_size) {
    if (partition_size <= 0) return units > 0 ? 1 : 0;
    const long long per = partition_size / unit;
    return (units + per - 1) / per;
}

// A partition size for units of `unit` tokens visible to each (sequence, kv
// head): as many partitions as leave every SM one deep thread block, of 256
// tokens at least; 0, one pass, where the sequences alone do.  A window over
// 16-bit pools, two sequences of 4 kv heads, 4096 tokens visible: one pass 14.7
// us, 17 partitions 8.9; 16 of 8 heads, 1024 visible: one pass 15.2, two
// partitions (more thread blocks than SMs, so wide ones) 22.
int choose_deep_partition(long long pairs, long long units, int unit) {
    if (pairs <= 0 || units <= 0) return 0;
    const long long parts = std::max(1, sm_count()) / pairs;
    if (parts < 2) return 0;
    const long long step = std::max(16, unit), tokens = units * unit;
    const long long size = std::max<long long>(((tokens + parts - 1) / parts + step - 1) / step * step, 256);
    return size >= tokens || size > INT_MAX / 2 ? 0 : static_cast<int>(size);
}

// 4-bit pools: the same while the SMs hold the (sequence, kv head) pairs twice
// (one 32k sequence of 8 heads: 15.9 us, 19.5 in wide blocks of 1024 tokens) or
// contexts are short; beyond, partitions for wide blocks: 2048 tokens (one's
// start and merge cost as much as 100 tokens a warp), more where that would be
// over 16 an SM.
int choose_int4_partition(long long pairs, long long units, int unit) {
    const long long sms = std::max(1, sm_count()), tokens = units * unit;
    if (2 * pairs <= sms || (pairs <= sms && tokens <= 4096)) return choose_deep_partition(pairs, units, unit);
    const long long work = tokens > LLONG_MAX / pairs ? LLONG_MAX : tokens * pairs;
    const long long size = (std::max<long long>(work / (16 * sms), 2048) + unit - 1) / unit * unit;
    return size >= tokens || size > INT_MAX / 2 ? 0 : static_cast<int>(size);
}

pa_status check_window(int window, int num_sinks, int least) {
    return window < least || num_sinks < 0 ? PA_ERR_INVALID_ARG : PA_OK;
}

// The partials' place: sets up p for `parts` partitions, or refuses.
pa_status take_workspace(pa::DecodeParams& p, const DecodeShape& sh, long long parts, void* workspace,
                         size_t workspace_bytes, int32_t* counters, int64_t num_counters) {
    p.num_partitions = static_cast<int>(parts);
    if (parts <= 1) return PA_OK;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < splitk_bytes(sh.num_seqs, sh.num_q_heads, parts, sh.head_dim))
        return PA_ERR_WORKSPACE;
    if (!counters || !aligned4(counters) ||
        num_counters < static_cast<int64_t>(sh.num_seqs) * sh.num_kv_heads)
        return PA_ERR_WORKSPACE;
    p.part_acc = static_cast<float*>(workspace);
    p.part_ml = p.part_acc + static_cast<size_t>(sh.num_seqs) * sh.num_q_heads * parts * sh.head_dim;
    p.counters = counters;
    return PA_OK;
}

template <bool FP8>
pa_status decode_window(void* out, const void* q, const void* key, const void* value, const void* k_cache,
                        const void* v_cache, const float* k_scale, const float* v_scale,
                        const int32_t* block_tables, const int32_t* context_lens, float scale, const DecodeShape& sh,
                        int window, int num_sinks, int partition_size, void* workspace, size_t workspace_bytes,
                        int32_t* counters, int64_t num_counters, const int32_t* ref_counts, const int32_t* seq_order,
                        void* stream) {
    pa_status st = check_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    if (st == PA_OK) st = check_scales<FP8>(sh, k_scale, v_scale);
    if (st == PA_OK) st = check_window(window, num_sinks, 1);
    if (st != PA_OK) return st;
    if (partition_size < 0 || partition_size % 16 != 0 || partition_size % sh.block_size != 0)
        return PA_ERR_INVALID_ARG;
    if ((key == nullptr) != (value == nullptr) || !aligned16(key) || !aligned16(value)) return PA_ERR_INVALID_ARG;
    if (!aligned4(seq_order) || !aligned4(ref_counts)) return PA_ERR_INVALID_ARG;
    if (sh.num_seqs == 0) return PA_OK;
    pa::DecodeParams p = make_params(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    p.seq_order = seq_order;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.new_key = key;
    p.new_value = value;
    p.ref_counts = ref_counts;
    p.window = window;
    p.num_sinks = num_sinks;
    const long long units = visible_units(p.context_cap, window, num_sinks, sh.block_size);
    const long long parts = window_partitions(units, sh.block_size, partition_size);
    if (parts > INT_MAX) return PA_ERR_UNSUPPORTED;
    st = take_workspace(p, sh, parts, workspace, workspace_bytes, counters, num_counters);
    if (st != PA_OK) return st;
    const pa_dtype dtype = static_cast<pa_dtype>(sh.dtype);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (parts > 1) {
        p.partition_blocks = partition_size / sh.block_size;
        const dim3 grid(static_cast<unsigned>(parts), sh.num_kv_heads, sh.num_seqs);
        e = decode_dispatch<true, FP8, false, true>(dtype, sh.head_dim, sh.block_size, p, grid, s);
    } else {
        const long long most = std::min<long long>(units * sh.block_size, INT_MAX);
        const dim3 grid = two_class_grid(p, dim3(1, sh.num_kv_heads, sh.num_seqs), static_cast<int>(most),
                                         sh.block_size);
        e = decode_dispatch<false, FP8, false, true>(dtype, sh.head_dim, sh.block_size, p, grid, s);
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Calls f(TypeTag<T>, IntTag<D>) for a row kernel's variant; the shape has been validated already.
template <typename F>
cudaError_t with_rows(pa_dtype dt, int D, F&& f) {
    auto by_dim = [&](auto tt) -> cudaError_t { return D == 64 ? f(tt, IntTag<64>{}) : f(tt, IntTag<128>{}); };
    switch (dt) {
        case PA_F32: return by_dim(TypeTag<float>{});
        case PA_F16: return by_dim(TypeTag<__half>{});
        default: return by_dim(TypeTag<__nv_bfloat16>{});
    }
}

int block_shift(int block_size) { return block_size == 8 ? 3 : (block_size == 16 ? 4 : 5); }

pa_status check_row_shape(int64_t num_tokens, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                          int dtype) {
    if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return PA_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// At most this many rows (tokens x kv heads) go one by one.  A write of 8 heads,
// one by one / by groups: 256 tokens 2.8 / 2.6 us in order, 2.8 / 6.4 at
// scattered slots; 512 tokens 3.7 / 2.7 and 3.7 / 6.4; 4096 tokens 13.4 / 6.8 and
// 13.4 / 16.5.  Scattered slots are a decode step's, seldom over 512 sequences.
constexpr long long kInt4FewRows = 4096;
template <bool WRITE>
pa_status rows_int4(void* key, void* value, void* k_cache, void* v_cache, const int64_t* slot_mapping,
                    int64_t num_tokens, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                    pa_dtype dtype, void* stream) {
    const pa_status st = check_row_shape(num_tokens, num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK || num_tokens == 0) return st;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned8(slot_mapping))
        return PA_ERR_INVALID_ARG;
    pa::RowsInt4Params p{};
    p.key = key;
    p.value = value;
    p.k_cache = static_cast<uint8_t*>(k_cache);
    p.v_cache = static_cast<uint8_t*>(v_cache);
    p.slot_mapping = slot_mapping;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.block_shift = block_shift(block_size);
    p.num_slots = num_blocks * static_cast<long long>(block_size);
    if (num_tokens > LLONG_MAX / 4096 / num_kv_heads) return PA_ERR_UNSUPPORTED;
    // Few rows go one by one, a thread for each 16-byte vector; many by groups
    // of a block's tokens, a warp for each.
    const bool rows = num_tokens * num_kv_heads <= kInt4FewRows;
    const int group = block_size == 8 ? 8 : 16;
    const long long blocks = rows ? (num_tokens * num_kv_heads * (head_dim * elem_size(dtype) / 16) + 255) / 256
                                  : ((num_tokens + group - 1) / group * num_kv_heads + 1) / 2;
    if (blocks > INT_MAX / 4) return PA_ERR_UNSUPPORTED;   // (the kernels' unit numbers fit 32 bits)
    const cudaError_t e = with_rows(dtype, head_dim, [&](auto tt, auto dd) -> cudaError_t {
        using T = typename decltype(tt)::type;
        constexpr int kD = decltype(dd)::value;
        auto kernel = rows ? pa::pa_rows_int4_kernel<T, kD, WRITE>
                           : (group == 8 ? pa::pa_groups_int4_kernel<T, kD, 8, WRITE>
                                         : pa::pa_groups_int4_kernel<T, kD, 16, WRITE>);
        return launch_early(kernel, dim3(static_cast<unsigned>(blocks)), dim3(rows ? 256 : 128), 0,
                            static_cast<cudaStream_t>(stream), PA_EARLY_LAUNCH, p);
    });
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Threads of a token's thread block: few tokens take 256, so that each is done
// sooner; many (8 an SM and more) take 64, which set up less and wait for one
// another less (6166 tokens of 48 rows, normed: 64 threads 37 us, 128 44, 32 43).
constexpr int kRopeManyThreads = 64;

template <pa::Pool POOL>
pa_status rope_and_cache(void* q_out, const void* q, const void* key, const void* value, void* k_cache, void* v_cache,
                         const float* k_scale, const float* v_scale, const int64_t* positions,
                         const int64_t* slot_mapping, const float* inv_freq, const void* q_weight,
                         const void* k_weight, float eps, float rope_scale, int interleaved, int rotary_dim,
                         int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t num_tokens, int num_q_heads,
                         int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, pa_dtype dtype,
                         void* stream) {
    const pa_status st = check_row_shape(num_tokens, num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK) return st;
    if (num_q_heads <= 0 || !std::isfinite(eps) || eps < 0.f || !std::isfinite(rope_scale)) return PA_ERR_INVALID_ARG;
    if (num_q_heads > INT_MAX / 4 || num_kv_heads > INT_MAX / 4) return PA_ERR_UNSUPPORTED;
    if (rotary_dim < 0 || rotary_dim > head_dim) return PA_ERR_INVALID_ARG;
    if (rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    const int per_vec = 16 / elem_size(dtype);
    if (q_stride < static_cast<int64_t>(num_q_heads) * head_dim ||
        k_stride < static_cast<int64_t>(num_kv_heads) * head_dim ||
        v_stride < static_cast<int64_t>(num_kv_heads) * head_dim || q_stride % per_vec || k_stride % per_vec ||
        v_stride % per_vec)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (num_tokens > INT_MAX) return PA_ERR_UNSUPPORTED;
    if (!q_out || !q || !key || !value || !k_cache || !v_cache || !positions || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (rotary_dim > 0 && !inv_freq) return PA_ERR_INVALID_ARG;
    if (!aligned16(q_out) || !aligned16(q) || !aligned16(key) || !aligned16(value) || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned8(positions) ||
        !aligned8(slot_mapping) || !aligned4(inv_freq))
        return PA_ERR_INVALID_ARG;
    if (POOL == pa::Pool::kE4m3 && (!k_scale || !v_scale || !aligned4(k_scale) || !aligned4(v_scale)))
        return PA_ERR_INVALID_ARG;
    pa::RopeParams p{};
    p.q_out = q_out;
    p.q = q;
    p.key = key;
    p.value = value;
    p.k_cache = static_cast<uint8_t*>(k_cache);
    p.v_cache = static_cast<uint8_t*>(v_cache);
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.inv_freq = inv_freq;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.rope_scale = rope_scale;
    p.eps = eps;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.rotary_dim = rotary_dim;
    p.block_shift = block_shift(block_size);
    p.num_slots = num_blocks * static_cast<long long>(block_size);
    const int threads = num_tokens >= 8LL * sm_count() ? kRopeManyThreads : pa::kRopeThreads;
    const cudaError_t e = with_rows(dtype, head_dim, [&](auto tt, auto dd) -> cudaError_t {
        using T = typename decltype(tt)::type;
        constexpr int kD = decltype(dd)::value;
        const bool norm = q_weight != nullptr || k_weight != nullptr;
        auto kernel = interleaved ? (norm ? pa::pa_rope_cache_kernel<T, kD, POOL, true, true>
                                          : pa::pa_rope_cache_kernel<T, kD, POOL, true, false>)
                                  : (norm ? pa::pa_rope_cache_kernel<T, kD, POOL, false, true>
                                          : pa::pa_rope_cache_kernel<T, kD, POOL, false, false>);
        return launch_early(kernel,
                            dim3(static_cast<unsigned>(num_tokens)), dim3(threads), 0,
                            static_cast<cudaStream_t>(stream), PA_EARLY_LAUNCH, p);
    });
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Thread blocks of the 4-bit decode: 4 warps, or 12 where the SMs hold one each
// of all of them (deep); each warp with a ring of 32-token stages (13.8 KB; 9/8
// bytes an element of K and V).
constexpr int kInt4WideWarps = 4, kInt4DeepWarps = 12;
constexpr int kInt4Step = 32;
template <int D>
constexpr int kInt4Stages = 13824 / (2 * pa::int4_tile_bytes(kInt4Step, D));

template <typename T, int D, int B, int NW>
cudaError_t launch_int4(const pa::DecodeParams& p, dim3 grid, cudaStream_t stream) {
    auto kernel = p.group <= 4 ? pa::pa_decode_int4_kernel<T, D, B, NW, kInt4Stages<D>, true>
                               : pa::pa_decode_int4_kernel<T, D, B, NW, kInt4Stages<D>, false>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
    return launch_early(kernel, grid, dim3(NW * 32), pa::Int4Smem<D, B, NW, kInt4Stages<D>>::kTotal, stream,
                        PA_EARLY_LAUNCH, p);
}

}  // namespace

extern "C" {

pa_status pa_rope_and_cache(void* q_out, const void* q, const void* key, const void* value, void* k_cache,
                            void* v_cache, const int64_t* positions, const int64_t* slot_mapping,
                            const float* inv_freq, const void* q_weight, const void* k_weight, float eps,
                            float rope_scale, int interleaved, int rotary_dim, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, int64_t num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                            int block_size, int64_t num_blocks, pa_dtype dtype, void* stream) {
    return rope_and_cache<pa::Pool::kNative>(q_out, q, key, value, k_cache, v_cache, nullptr, nullptr, positions,
                                             slot_mapping, inv_freq, q_weight, k_weight, eps, rope_scale, interleaved,
                                             rotary_dim, q_stride, k_stride, v_stride, num_tokens, num_q_heads,
                                             num_kv_heads, head_dim, block_size, num_blocks, dtype, stream);
}

pa_status pa_rope_and_cache_fp8(void* q_out, const void* q, const void* key, const void* value, void* k_cache,
                                void* v_cache, const float* k_scale, const float* v_scale, const int64_t* positions,
                                const int64_t* slot_mapping, const float* inv_freq, const void* q_weight,
                                const void* k_weight, float eps, float rope_scale, int interleaved, int rotary_dim,
                                int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t num_tokens,
                                int num_q_heads, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                                pa_dtype dtype, void* stream) {
    return rope_and_cache<pa::Pool::kE4m3>(q_out, q, key, value, k_cache, v_cache, k_scale, v_scale, positions,
                                           slot_mapping, inv_freq, q_weight, k_weight, eps, rope_scale, interleaved,
                                           rotary_dim, q_stride, k_stride, v_stride, num_tokens, num_q_heads,
                                           num_kv_heads, head_dim, block_size, num_blocks, dtype, stream);
}

pa_status pa_rope_and_cache_int4(void* q_out, const void* q, const void* key, const void* value, void* k_cache,
                                 void* v_cache, const int64_t* positions, const int64_t* slot_mapping,
                                 const float* inv_freq, const void* q_weight, const void* k_weight, float eps,
                                 float rope_scale, int interleaved, int rotary_dim, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, int64_t num_tokens, int num_q_heads,
                                 int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, pa_dtype dtype,
                                 void* stream) {
    return rope_and_cache<pa::Pool::kInt4>(q_out, q, key, value, k_cache, v_cache, nullptr, nullptr, positions,
                                           slot_mapping, inv_freq, q_weight, k_weight, eps, rope_scale, interleaved,
                                           rotary_dim, q_stride, k_stride, v_stride, num_tokens, num_q_heads,
                                           num_kv_heads, head_dim, block_size, num_blocks, dtype, stream);
}

pa_status pa_reshape_and_cache_int4(const void* key, const void* value, void* k_cache, void* v_cache,
                                    const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads, int head_dim,
                                    int block_size, int64_t num_blocks, pa_dtype dtype, void* stream) {
    return rows_int4<true>(const_cast<void*>(key), const_cast<void*>(value), k_cache, v_cache, slot_mapping,
                           num_tokens, num_kv_heads, head_dim, block_size, num_blocks, dtype, stream);
}

pa_status pa_gather_cache_int4(void* key, void* value, const void* k_cache, const void* v_cache,
                               const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads, int head_dim,
                               int block_size, int64_t num_blocks, pa_dtype dtype, void* stream) {
    return rows_int4<false>(key, value, const_cast<void*>(k_cache), const_cast<void*>(v_cache), slot_mapping,
                            num_tokens, num_kv_heads, head_dim, block_size, num_blocks, dtype, stream);
}

pa_status pa_decode_int4_plan(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_context_len,
                              int window, int num_sinks, int* partition_size, size_t* bytes) {
    if (!partition_size || !bytes || num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_context_len < 0 || *partition_size < -1 || check_window(window, num_sinks, 0) != PA_OK)
        return PA_ERR_INVALID_ARG;
    const long long units = visible_units(max_context_len, window, num_sinks, kInt4Step);
    if (*partition_size < 0)
        *partition_size = choose_int4_partition(static_cast<long long>(num_seqs) * num_kv_heads, units, kInt4Step);
    if (*partition_size % kInt4Step != 0) return PA_ERR_INVALID_ARG;
    const long long parts = window_partitions(units, kInt4Step, *partition_size);
    *bytes = parts > 1 ? splitk_bytes(num_seqs, num_q_heads, parts, head_dim) : 0;
    return PA_OK;
}

pa_status pa_decode_int4(void* out, const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_tables, const int32_t* context_lens, float scale, int block_size,
                         int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                         int max_context_len, int64_t num_blocks, pa_dtype dtype, int window, int num_sinks,
                         int partition_size, void* workspace, size_t workspace_bytes, int32_t* counters,
                         int64_t num_counters, const int32_t* seq_order, void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    pa_status st = check_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    if (st == PA_OK) st = check_window(window, num_sinks, 0);
    if (st != PA_OK) return st;
    if (dtype == PA_F32) return PA_ERR_UNSUPPORTED;  // 4-bit pools take 16-bit queries
    if (partition_size < 0 || partition_size % kInt4Step != 0) return PA_ERR_INVALID_ARG;
    if (!aligned4(seq_order)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    pa::DecodeParams p = make_params(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    p.seq_order = seq_order;
    p.window = window;
    p.num_sinks = num_sinks;
    const long long units = visible_units(p.context_cap, window, num_sinks, kInt4Step);
    const long long parts = window_partitions(units, kInt4Step, partition_size);
    if (parts > INT_MAX) return PA_ERR_UNSUPPORTED;
    st = take_workspace(p, sh, parts, workspace, workspace_bytes, counters, num_counters);
    if (st != PA_OK) return st;
    p.partition_blocks = parts > 1 ? partition_size / kInt4Step : INT_MAX / 2;
    const dim3 grid(static_cast<unsigned>(std::max(1LL, parts)), num_kv_heads, num_seqs);
    const bool deep = std::max(1LL, parts) * num_kv_heads * num_seqs <= sm_count();
    const cudaError_t e = with_variant(dtype, head_dim, block_size, [&](auto tt, auto dd, auto bb) -> cudaError_t {
        using T = typename decltype(tt)::type;
        constexpr int kD = decltype(dd)::value, kB = decltype(bb)::value;
        if constexpr (pa::IsF32<T>::value) {
            return cudaErrorInvalidValue;
        } else {
            return deep ? launch_int4<T, kD, kB, kInt4DeepWarps>(p, grid, static_cast<cudaStream_t>(stream))
                        : launch_int4<T, kD, kB, kInt4WideWarps>(p, grid, static_cast<cudaStream_t>(stream));
        }
    });
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_decode_window_plan(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                int max_context_len, int window, int num_sinks, int* partition_size, size_t* bytes) {
    if (!partition_size || !bytes || num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        block_size <= 0 || max_context_len < 0 || *partition_size < -1 ||
        check_window(window, num_sinks, 1) != PA_OK)
        return PA_ERR_INVALID_ARG;
    const long long units = visible_units(max_context_len, window, num_sinks, block_size);
    if (*partition_size < 0)
        *partition_size = choose_deep_partition(static_cast<long long>(num_seqs) * num_kv_heads, units, block_size);
    if (*partition_size % 16 != 0 || *partition_size % block_size != 0) return PA_ERR_INVALID_ARG;
    const long long parts = window_partitions(units, block_size, *partition_size);
    *bytes = parts > 1 ? splitk_bytes(num_seqs, num_q_heads, parts, head_dim) : 0;
    return PA_OK;
}

pa_status pa_decode_window(void* out, const void* q, const void* key, const void* value, void* k_cache, void* v_cache,
                           const int32_t* block_tables, const int32_t* context_lens, float scale, int block_size,
                           int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                           int max_context_len, int64_t num_blocks, pa_dtype dtype, int window, int num_sinks,
                           int partition_size, void* workspace, size_t workspace_bytes, int32_t* counters,
                           int64_t num_counters, const int32_t* ref_counts, const int32_t* seq_order, void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    return decode_window<false>(out, q, key, value, k_cache, v_cache, nullptr, nullptr, block_tables, context_lens,
                                scale, sh, window, num_sinks, partition_size, workspace, workspace_bytes, counters,
                                num_counters, ref_counts, seq_order, stream);
}

pa_status pa_decode_window_fp8(void* out, const void* q, const void* key, const void* value, void* k_cache,
                               void* v_cache, const float* k_scale, const float* v_scale,
                               const int32_t* block_tables, const int32_t* context_lens, float scale, int block_size,
                               int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                               int max_context_len, int64_t num_blocks, pa_dtype dtype, int window, int num_sinks,
                               int partition_size, void* workspace, size_t workspace_bytes, int32_t* counters,
                               int64_t num_counters, const int32_t* ref_counts, const int32_t* seq_order,
                               void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    return decode_window<true>(out, q, key, value, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                               scale, sh, window, num_sinks, partition_size, workspace, workspace_bytes, counters,
                               num_counters, ref_counts, seq_order, stream);
}

pa_status pa_prefill_window(void* out, const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
                            float scale, int block_size, int num_seqs, int num_q_heads, int num_kv_heads,
                            int head_dim, int max_blocks_per_seq, int max_context_len, int max_query_len,
                            int64_t num_blocks, pa_dtype dtype, int window, int num_sinks, void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    pa_status st = check_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    if (st == PA_OK) st = check_window(window, num_sinks, 1);
    if (st != PA_OK) return st;
    if (dtype == PA_F32) return PA_ERR_UNSUPPORTED;  // the tensor-core path takes 16-bit inputs
    if (scale <= 0.f || max_query_len < 0) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || max_query_len == 0) return PA_OK;
    if (!query_start || !aligned4(query_start)) return PA_ERR_INVALID_ARG;
    CUtensorMap k_rows{};
    if (!prefill_k_source(&k_rows, k_cache, dtype, block_size, head_dim, num_kv_heads, num_blocks))
        return PA_ERR_UNSUPPORTED;
    pa::PrefillParams p{};
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.score_scale = scale * 1.4426950408889634f;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_cap = context_cap(sh);
    p.num_blocks = num_blocks;
    p.tile_tokens = 128 / p.group;
    // (no more than the context: the kernel's differences of positions stay within 32 bits)
    p.window = std::min(window, std::max(1, p.context_cap));
    p.num_sinks = std::min(num_sinks, p.context_cap);
    const long long per_cta = static_cast<long long>(prefill_tiles_per_cta(block_size, false)) * p.tile_tokens;
    const long long tiles = (static_cast<long long>(max_query_len) + per_cta - 1) / per_cta;
    if (tiles > INT_MAX) return PA_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(tiles), num_kv_heads, num_seqs);
    const cudaError_t e = with_variant(dtype, head_dim, block_size, [&](auto tt, auto dd, auto bb) -> cudaError_t {
        using T = typename decltype(tt)::type;
        constexpr int kD = decltype(dd)::value, kB = decltype(bb)::value;
        if constexpr (pa::IsF32<T>::value) {
            return cudaErrorInvalidValue;
        } else {
            return launch_prefill_tc<T, kD, kB, false, true>(p, k_rows, grid, static_cast<cudaStream_t>(stream));
        }
    });
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"

// This unit's device error word, read and cleared (the stream has been synchronised).
extern "C" __attribute__((visibility("hidden"))) cudaError_t pa_ops_take_error(int* value) {
    cudaError_t e = cudaMemcpyFromSymbol(value, pa::g_device_error, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *value != 0) e = cudaMemcpyToSymbol(pa::g_device_error, &zero, sizeof(int));
    return e;
}

#ifdef PA_TEST_HOOKS
// This unit's copies of the test hooks (pa_test_set_hooks sets both units').
extern "C" __attribute__((visibility("hidden"))) cudaError_t pa_ops_set_hooks(unsigned long long limit_ns,
                                                                             int skip_first_copy) {
    const cudaError_t e = cudaMemcpyToSymbol(pa::g_test_wait_limit_ns, &limit_ns, sizeof(limit_ns));
    return e != cudaSuccess ? e : cudaMemcpyToSymbol(pa::g_test_skip_first_copy, &skip_first_copy, sizeof(int));
}
#endif  // PA_TEST_HOOKS
