// Host side of the C ABI declared in include/pa.h: argument validation,
// kernel-variant dispatch on (dtype, head_dim, block_size), launches.
// Nothing here allocates device memory or synchronises, except
// pa_get_device_error which synchronises the given stream by contract.

#include "pa_host.cuh"

#include "pa_blocks.cuh"
#include "pa_copy.cuh"
#include "pa_reshape.cuh"

// The error word of the other translation unit (pa_ops.cu), read and cleared.
extern "C" __attribute__((visibility("hidden"))) cudaError_t pa_ops_take_error(int* value);

extern "C" {

pa_status pa_reshape_and_cache(const void* key, const void* value, void* k_cache, void* v_cache,
                               const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads,
                               int head_dim, int block_size, int64_t num_blocks, pa_dtype dtype,
                               void* stream) {
    if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return PA_ERR_UNSUPPORTED;
    const int row_bytes = head_dim * elem_size(dtype);
    if (row_bytes % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PA_ERR_INVALID_ARG;
    pa::ReshapeParams p{};
    p.key = static_cast<const uint4*>(key);
    p.value = static_cast<const uint4*>(value);
    p.k_cache = static_cast<uint4*>(k_cache);
    p.v_cache = static_cast<uint4*>(v_cache);
    p.slot_mapping = slot_mapping;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.vecs_per_row = row_bytes / 16;
    p.block_size = block_size;
    p.num_slots = num_blocks * static_cast<long long>(block_size);
    const long long threads = num_tokens * num_kv_heads * static_cast<long long>(p.vecs_per_row);
    const long long blocks = (threads + 255) / 256;
    if (blocks > INT_MAX) return PA_ERR_UNSUPPORTED;
    return launch_early(pa::pa_reshape_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                        static_cast<cudaStream_t>(stream), PA_EARLY_LAUNCH, p) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status pa_decode(void* out, const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* block_tables, const int32_t* context_lens, float scale, int block_size,
                    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                    int max_context_len, int64_t num_blocks, pa_dtype dtype, const int32_t* seq_order,
                    void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    return decode_one_pass<false>(out, q, k_cache, v_cache, nullptr, nullptr, block_tables, context_lens, scale, sh,
                                  seq_order, stream);
}

pa_status pa_decode_append(void* out, const void* q, const void* key, const void* value, void* k_cache, void* v_cache,
                           const int32_t* block_tables, const int32_t* context_lens, float scale, int block_size,
                           int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                           int max_context_len, int64_t num_blocks, pa_dtype dtype, const int32_t* ref_counts,
                           const int32_t* seq_order, void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    pa_status st = check_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    if (st != PA_OK || num_seqs == 0) return st;
    if (!key || !value || !aligned16(key) || !aligned16(value)) return PA_ERR_INVALID_ARG;
    if (!aligned4(seq_order) || !aligned4(ref_counts)) return PA_ERR_INVALID_ARG;
    pa::DecodeParams p = make_params(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    p.seq_order = seq_order;
    p.new_key = key;
    p.new_value = value;
    p.ref_counts = ref_counts;
    const dim3 grid = two_class_grid(p, dim3(1, num_kv_heads, num_seqs), max_context_len, block_size);
    const cudaError_t e = decode_dispatch<false>(dtype, head_dim, block_size, p, grid,
                                                 static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_decode_splitk_workspace_size(int num_seqs, int num_q_heads, int head_dim, int max_context_len,
                                          int partition_size, size_t* bytes) {
    if (!bytes || num_seqs < 0 || num_q_heads <= 0 || head_dim <= 0 || max_context_len < 0 ||
        partition_size <= 0)
        return PA_ERR_INVALID_ARG;
    const long long parts = (static_cast<long long>(max_context_len) + partition_size - 1) / partition_size;
    *bytes = splitk_bytes(num_seqs, num_q_heads, parts, head_dim);
    return PA_OK;
}

pa_status pa_decode_splitk(void* out, const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_tables, const int32_t* context_lens, float scale,
                           int block_size, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                           int max_blocks_per_seq, int max_context_len, int64_t num_blocks, pa_dtype dtype,
                           int partition_size, void* workspace, size_t workspace_bytes, int32_t* counters,
                           int64_t num_counters, const int32_t* seq_order, void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    return decode_split<false>(out, q, k_cache, v_cache, nullptr, nullptr, block_tables, context_lens, scale, sh,
                               partition_size, workspace, workspace_bytes, counters, num_counters, seq_order,
                               stream);
}

pa_status pa_reshape_and_cache_fp8(const void* key, const void* value, void* k_cache, void* v_cache,
                                   const int64_t* slot_mapping, const float* k_scale, const float* v_scale,
                                   int64_t num_tokens, int num_kv_heads, int head_dim, int block_size,
                                   int64_t num_blocks, pa_dtype dtype, void* stream) {
    if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return PA_ERR_UNSUPPORTED;
    if (head_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping || !k_scale || !v_scale) return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) || !aligned4(k_scale) || !aligned4(v_scale))
        return PA_ERR_INVALID_ARG;
    if (block_size != 8 && block_size % 16 != 0) return PA_ERR_UNSUPPORTED;
    pa::ReshapeE4m3Params p{};
    p.key = key;
    p.value = value;
    p.k_cache = static_cast<uint32_t*>(k_cache);
    p.v_cache = static_cast<uint8_t*>(v_cache);
    p.slot_mapping = slot_mapping;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.num_tokens = num_tokens;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.block_size = block_size;
    p.num_slots = num_blocks * static_cast<long long>(block_size);
    const long long threads = num_tokens * num_kv_heads * static_cast<long long>(head_dim / 4);
    const long long blocks = (threads + 255) / 256;
    if (blocks > INT_MAX) return PA_ERR_UNSUPPORTED;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned g = static_cast<unsigned>(blocks);
    cudaError_t e;
    switch (dtype) {
        case PA_F32: e = launch_early(pa::pa_reshape_e4m3_kernel<float>, dim3(g), dim3(256), 0, st, PA_EARLY_LAUNCH, p); break;
        case PA_F16: e = launch_early(pa::pa_reshape_e4m3_kernel<__half>, dim3(g), dim3(256), 0, st, PA_EARLY_LAUNCH, p); break;
        default:
            e = launch_early(pa::pa_reshape_e4m3_kernel<__nv_bfloat16>, dim3(g), dim3(256), 0, st, PA_EARLY_LAUNCH, p);
            break;
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_decode_fp8(void* out, const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                        const float* v_scale, const int32_t* block_tables, const int32_t* context_lens, float scale,
                        int block_size, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                        int max_blocks_per_seq, int max_context_len, int64_t num_blocks, pa_dtype dtype,
                        const int32_t* seq_order, void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    return decode_one_pass<true>(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale, sh,
                                 seq_order, stream);
}

pa_status pa_decode_append_fp8(void* out, const void* q, const void* key, const void* value, void* k_cache,
                               void* v_cache, const float* k_scale, const float* v_scale, const int32_t* block_tables,
                               const int32_t* context_lens, float scale, int block_size, int num_seqs,
                               int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                               int max_context_len, int64_t num_blocks, pa_dtype dtype,
                               const int32_t* ref_counts, const int32_t* seq_order, void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    if (num_seqs > 0 && (!key || !value || !aligned16(key) || !aligned16(value))) return PA_ERR_INVALID_ARG;
    if (!aligned4(ref_counts)) return PA_ERR_INVALID_ARG;
    return decode_one_pass<true>(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale, sh,
                                 seq_order, stream, key, value, ref_counts);
}

pa_status pa_decode_splitk_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, const int32_t* block_tables,
                               const int32_t* context_lens, float scale, int block_size, int num_seqs,
                               int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                               int max_context_len, int64_t num_blocks, pa_dtype dtype, int partition_size,
                               void* workspace, size_t workspace_bytes, int32_t* counters, int64_t num_counters,
                               const int32_t* seq_order, void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    return decode_split<true>(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale, sh,
                              partition_size, workspace, workspace_bytes, counters, num_counters, seq_order, stream);
}

pa_status pa_copy_blocks(void* dst_k_cache, void* dst_v_cache, const void* src_k_cache, const void* src_v_cache,
                         const int64_t* block_mapping, int64_t num_pairs, int num_kv_heads, int head_dim,
                         int block_size, int64_t src_num_blocks, int64_t dst_num_blocks, pa_dtype dtype,
                         void* stream) {
    if (num_pairs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || src_num_blocks <= 0 ||
        dst_num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return PA_ERR_UNSUPPORTED;
    const long long block_bytes =
        static_cast<long long>(num_kv_heads) * block_size * head_dim * elem_size(dtype);
    if ((static_cast<long long>(head_dim) * elem_size(dtype)) % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (num_pairs == 0) return PA_OK;
    if (!dst_k_cache || !dst_v_cache || !src_k_cache || !src_v_cache || !block_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(dst_k_cache) || !aligned16(dst_v_cache) || !aligned16(src_k_cache) ||
        !aligned16(src_v_cache) || (reinterpret_cast<uintptr_t>(block_mapping) & 7u))
        return PA_ERR_INVALID_ARG;
    if (!device_accessible(dst_k_cache) || !device_accessible(dst_v_cache) || !device_accessible(src_k_cache) ||
        !device_accessible(src_v_cache) || !device_accessible(block_mapping))
        return PA_ERR_INVALID_ARG;
    pa::CopyParams p{};
    p.dst[0] = static_cast<uint4*>(dst_k_cache);
    p.dst[1] = static_cast<uint4*>(dst_v_cache);
    p.src[0] = static_cast<const uint4*>(src_k_cache);
    p.src[1] = static_cast<const uint4*>(src_v_cache);
    p.mapping = block_mapping;
    p.num_pairs = num_pairs;
    p.vecs_per_block = block_bytes / 16;
    p.src_blocks = src_num_blocks;
    p.dst_blocks = dst_num_blocks;
    p.chunks = static_cast<int>((p.vecs_per_block + pa::kChunkVecs - 1) / pa::kChunkVecs);
    const long long ctas = num_pairs * 2 * p.chunks;
    if (ctas > INT_MAX) return PA_ERR_UNSUPPORTED;
    return launch_early(pa::pa_copy_blocks_kernel, dim3(static_cast<unsigned>(ctas)), dim3(pa::kCopyThreads), 0,
                        static_cast<cudaStream_t>(stream), PA_EARLY_LAUNCH, p) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status pa_prefill(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                     const int32_t* context_lens, const int32_t* query_start, float scale, int block_size,
                     int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_blocks_per_seq,
                     int max_context_len, int max_query_len, int64_t num_blocks, pa_dtype dtype, void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    pa_status st = check_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    if (st != PA_OK) return st;
    if (dtype == PA_F32) return PA_ERR_UNSUPPORTED;  // the tensor-core path takes 16-bit inputs
    if (max_query_len < 0) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || max_query_len == 0) return PA_OK;
    if (!query_start || !aligned4(query_start)) return PA_ERR_INVALID_ARG;
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
    CUtensorMap k_rows{};
    const bool use_tc = PA_PREFILL_TC &&
                        prefill_k_source(&k_rows, k_cache, dtype, block_size, head_dim, num_kv_heads, num_blocks);
    p.tile_tokens = (use_tc ? 128 : kPrefillWarps * 16) / p.group;
    // the tensor-core kernel takes one or two query tiles per CTA
    const long long per_cta =
        use_tc ? static_cast<long long>(prefill_tiles_per_cta(block_size, false)) * p.tile_tokens : p.tile_tokens;
    const long long tiles = (static_cast<long long>(max_query_len) + per_cta - 1) / per_cta;
    if (tiles > INT_MAX) return PA_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(tiles), num_kv_heads, num_seqs);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = with_variant(dtype, head_dim, block_size, [&](auto tt, auto dd, auto bb) -> cudaError_t {
        using T = typename decltype(tt)::type;
        constexpr int kD = decltype(dd)::value, kB = decltype(bb)::value;
        if constexpr (pa::IsF32<T>::value) {
            return cudaErrorInvalidValue;
        } else {
            return use_tc ? launch_prefill_tc<T, kD, kB>(p, k_rows, grid, s) : launch_prefill<T, kD, kB>(p, grid, s);
        }
    });
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_decode_shared_prefix_workspace_size(int num_seqs, int num_q_heads, int head_dim, int prefix_blocks,
                                                 int block_size, size_t* bytes) {
    if (!bytes || num_seqs < 0 || num_q_heads <= 0 || head_dim <= 0 || prefix_blocks <= 0 || block_size <= 0)
        return PA_ERR_INVALID_ARG;
    *bytes = splitk_bytes(num_seqs, num_q_heads, shared_prefix_tiles(prefix_blocks, block_size) + 1, head_dim);
    return PA_OK;
}

pa_status pa_decode_shared_prefix(void* out, const void* q, const void* key, const void* value, void* k_cache,
                                  void* v_cache, const int32_t* block_tables, const int32_t* context_lens,
                                  float scale, int block_size, int num_seqs, int num_q_heads, int num_kv_heads,
                                  int head_dim, int max_blocks_per_seq, int max_context_len, int64_t num_blocks,
                                  pa_dtype dtype, int prefix_blocks, void* workspace, size_t workspace_bytes,
                                  int32_t* counters, int64_t num_counters, const int32_t* ref_counts,
                                  void* stream) {
    const DecodeShape sh{block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                         max_context_len, num_blocks, static_cast<int>(dtype)};
    pa_status st = check_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    if (st != PA_OK) return st;
    if (dtype == PA_F32) return PA_ERR_UNSUPPORTED;  // the prefix pass runs on the tensor cores
    if (prefix_blocks <= 0 || prefix_blocks > max_blocks_per_seq ||
        static_cast<long long>(prefix_blocks) * block_size > max_context_len)
        return PA_ERR_INVALID_ARG;
    if ((key == nullptr) != (value == nullptr)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (key && (!aligned16(key) || !aligned16(value))) return PA_ERR_INVALID_ARG;
    if (!aligned4(ref_counts)) return PA_ERR_INVALID_ARG;
    const int tiles = shared_prefix_tiles(prefix_blocks, block_size);
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < splitk_bytes(num_seqs, num_q_heads, tiles + 1, head_dim))
        return PA_ERR_WORKSPACE;
    if (!counters || !aligned4(counters) || num_counters < static_cast<int64_t>(num_seqs) * num_kv_heads)
        return PA_ERR_WORKSPACE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap k_rows{};
    if (!PA_PREFILL_TC ||
        !prefill_k_source(&k_rows, k_cache, dtype, block_size, head_dim, num_kv_heads, num_blocks)) {
        // no tensor map for the prefix pass: the plain decode gives the same result
        pa::DecodeParams p = make_params(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
        p.new_key = key;
        p.new_value = value;
        p.ref_counts = ref_counts;
        const dim3 grid = two_class_grid(p, dim3(1, num_kv_heads, num_seqs), max_context_len, block_size);
        return decode_dispatch<false>(dtype, head_dim, block_size, p, grid, s) == cudaSuccess ? PA_OK
                                                                                               : PA_ERR_CUDA;
    }
    // Pass 1 (tensor cores): the prefix once per kv head for all sequences,
    // key partitions spread over the SMs, unnormalised partials to the workspace.
    const int group = num_q_heads / num_kv_heads;
    const int tile_tokens = 128 / group;
    const int qt = prefill_tiles_per_cta(block_size, true);
    const long long row_ctas = (static_cast<long long>(num_seqs) + qt * tile_tokens - 1) / (qt * tile_tokens);
    const long long per_part = row_ctas * num_kv_heads;
    long long want = (PA_PREFIX_CTAS > 0 ? PA_PREFIX_CTAS : sm_count() / 3) / per_part;
    want = want < 1 ? 1 : (want > tiles ? tiles : want);
    const int tiles_per = static_cast<int>((tiles + want - 1) / want);
    const int parts = (tiles + tiles_per - 1) / tiles_per;   // every partition holds >= 1 tile (<= tiles)
    const int slots = parts + 1;                               // + the sequence's own blocks
    float* acc = static_cast<float*>(workspace);
    float* ml = acc + static_cast<size_t>(num_seqs) * num_q_heads * slots * head_dim;
    pa::PrefillParams pp{};
    pp.out = out;
    pp.context_lens = context_lens;
    pp.counters = counters;
    pp.prefix_append = key != nullptr;
    pp.q = q;
    pp.k_cache = k_cache;
    pp.v_cache = v_cache;
    pp.block_tables = block_tables;
    pp.score_scale = scale * 1.4426950408889634f;
    pp.num_seqs = num_seqs;
    pp.num_q_heads = num_q_heads;
    pp.num_kv_heads = num_kv_heads;
    pp.group = group;
    pp.max_blocks_per_seq = max_blocks_per_seq;
    pp.context_cap = context_cap(sh);
    pp.num_blocks = num_blocks;
    pp.tile_tokens = tile_tokens;
    pp.part_acc = acc;
    pp.part_ml = ml;
    pp.num_partitions = slots;
    pp.prefix_len = prefix_blocks * block_size;
    pp.prefix_tiles = tiles_per;
    const dim3 pgrid(static_cast<unsigned>(row_ctas), num_kv_heads, parts);
    cudaError_t e = with_variant(dtype, head_dim, block_size, [&](auto tt, auto dd, auto bb) -> cudaError_t {
        using T = typename decltype(tt)::type;
        constexpr int kD = decltype(dd)::value, kB = decltype(bb)::value;
        if constexpr (pa::IsF32<T>::value) {
            return cudaErrorInvalidValue;
        } else {
            return launch_prefill_tc<T, kD, kB, true>(pp, k_rows, pgrid, s);
        }
    });
    if (e != cudaSuccess) return PA_ERR_CUDA;
    // Pass 2: each sequence's own blocks (and newest token), the prefix
    // partials folded into the same merge.
    pa::DecodeParams p = make_params(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    p.new_key = key;
    p.new_value = value;
    p.ref_counts = ref_counts;
    p.part_acc = acc;
    p.part_ml = ml;
    p.first_block = prefix_blocks;
    p.num_partitions = slots;
    p.counters = counters;
    const int pre = prefix_blocks * block_size;
    const dim3 grid = two_class_grid(p, dim3(1, num_kv_heads, num_seqs), max_context_len, block_size,
                                     PA_PREFIX_CLASS_EIGHTHS > 0
                                         ? pre + static_cast<int>((static_cast<long long>(max_context_len - pre) *
                                                                   PA_PREFIX_CLASS_EIGHTHS) / 8)
                                         : 0);
    e = decode_dispatch<false, false, true>(dtype, head_dim, block_size, p, grid, s);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"

// ---- block management (pa_blocks.cuh)

namespace {

pa_status check_block_state(const int32_t* ref_counts, const int32_t* free_ids, const int64_t* free_state,
                            int64_t num_blocks) {
    if (num_blocks <= 0 || num_blocks > INT_MAX) return PA_ERR_INVALID_ARG;
    if (!ref_counts || !free_ids || !free_state) return PA_ERR_INVALID_ARG;
    if (!aligned4(ref_counts) || !aligned4(free_ids) || !aligned8(free_state)) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

pa_status check_rows(const int32_t* block_tables, const int32_t* context_lens, int num_seqs, int max_blocks_per_seq,
                     int block_size) {
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || block_size <= 0) return PA_ERR_INVALID_ARG;
    if (static_cast<long long>(max_blocks_per_seq) * block_size > INT_MAX) return PA_ERR_UNSUPPORTED;
    if (num_seqs > 0 && (!block_tables || !context_lens || !aligned4(block_tables) || !aligned4(context_lens)))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

pa::BlockState block_state(int32_t* ref_counts, const int32_t* free_ids, int64_t* free_state, int64_t num_blocks) {
    pa::BlockState st{};
    st.ref = ref_counts;
    st.free_ids = const_cast<int32_t*>(free_ids);
    st.free_state = reinterpret_cast<long long*>(free_state);
    st.num_blocks = num_blocks;
    return st;
}

}  // namespace

extern "C" {

pa_status pa_blocks_init(int32_t* ref_counts, int32_t* free_ids, int64_t* free_state, int64_t num_blocks,
                         void* stream) {
    const pa_status st = check_block_state(ref_counts, free_ids, free_state, num_blocks);
    if (st != PA_OK) return st;
    const long long blocks = std::min<long long>((num_blocks + 255) / 256, 4096);
    return launch_early(pa::pa_blocks_init_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                        static_cast<cudaStream_t>(stream), PA_EARLY_LAUNCH,
                        block_state(ref_counts, free_ids, free_state, num_blocks)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status pa_blocks_append(int32_t* block_tables, int32_t* context_lens, const int32_t* num_new_tokens,
                           int32_t* ref_counts, const int32_t* free_ids, int64_t* free_state, int64_t* slot_mapping,
                           int64_t num_slots, int64_t* copy_pairs, int num_seqs, int max_blocks_per_seq,
                           int block_size, int64_t num_blocks, void* stream) {
    pa_status st = check_block_state(ref_counts, free_ids, free_state, num_blocks);
    if (st == PA_OK) st = check_rows(block_tables, context_lens, num_seqs, max_blocks_per_seq, block_size);
    if (st != PA_OK) return st;
    if (num_slots < 0) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!num_new_tokens || !copy_pairs || !aligned4(num_new_tokens) || !aligned8(copy_pairs)) return PA_ERR_INVALID_ARG;
    if (num_slots > 0 && (!slot_mapping || !aligned8(slot_mapping))) return PA_ERR_INVALID_ARG;
    pa::AppendParams p{};
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.num_new = num_new_tokens;
    p.st = block_state(ref_counts, free_ids, free_state, num_blocks);
    p.slots = reinterpret_cast<long long*>(slot_mapping);
    p.num_slots = num_slots;
    p.pairs = reinterpret_cast<long long*>(copy_pairs);
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = block_size;
    const int threads = std::min(pa::kBlocksThreads, (num_seqs + 31) / 32 * 32);
    return launch_early(pa::pa_blocks_append_kernel, dim3(1), dim3(threads), 0, static_cast<cudaStream_t>(stream),
                        PA_EARLY_LAUNCH, p) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status pa_blocks_fork(int32_t* block_tables, int32_t* context_lens, int32_t* ref_counts, const int32_t* forks,
                         int num_forks, int num_seqs, int max_blocks_per_seq, int block_size, int64_t num_blocks,
                         void* stream) {
    pa_status st = check_rows(block_tables, context_lens, num_seqs, max_blocks_per_seq, block_size);
    if (st != PA_OK) return st;
    if (num_forks < 0 || num_blocks <= 0 || num_blocks > INT_MAX) return PA_ERR_INVALID_ARG;
    if (num_forks == 0 || num_seqs == 0) return PA_OK;
    if (!ref_counts || !forks || !aligned4(ref_counts) || !aligned4(forks)) return PA_ERR_INVALID_ARG;
    pa::ForkParams p{};
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.ref = ref_counts;
    p.forks = forks;
    p.num_forks = num_forks;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    return launch_early(pa::pa_blocks_fork_kernel, dim3(1), dim3(pa::kBlocksThreads), 0,
                        static_cast<cudaStream_t>(stream), PA_EARLY_LAUNCH, p) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status pa_blocks_release(int32_t* block_tables, int32_t* context_lens, int32_t* ref_counts, int32_t* free_ids,
                            int64_t* free_state, const int32_t* seqs, int num_release, int num_seqs,
                            int max_blocks_per_seq, int block_size, int64_t num_blocks, void* stream) {
    pa_status st = check_block_state(ref_counts, free_ids, free_state, num_blocks);
    if (st == PA_OK) st = check_rows(block_tables, context_lens, num_seqs, max_blocks_per_seq, block_size);
    if (st != PA_OK) return st;
    if (num_release < 0) return PA_ERR_INVALID_ARG;
    if (num_release == 0 || num_seqs == 0) return PA_OK;
    if (!seqs || !aligned4(seqs)) return PA_ERR_INVALID_ARG;
    pa::ReleaseParams p{};
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.st = block_state(ref_counts, free_ids, free_state, num_blocks);
    p.seqs = seqs;
    p.num_release = num_release;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = block_size;
    return launch_early(pa::pa_blocks_release_kernel, dim3(1), dim3(pa::kBlocksThreads), 0,
                        static_cast<cudaStream_t>(stream), PA_EARLY_LAUNCH, p) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status pa_get_device_error(void* stream, int32_t* code) {
    if (!code) return PA_ERR_INVALID_ARG;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return PA_ERR_CUDA;
    int value = 0;
    if (cudaMemcpyFromSymbol(&value, pa::g_device_error, sizeof(int)) != cudaSuccess) return PA_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(pa::g_device_error, &zero, sizeof(int)) != cudaSuccess) return PA_ERR_CUDA;
    int other = 0;
    if (pa_ops_take_error(&other) != cudaSuccess) return PA_ERR_CUDA;
    *code = value | other;
    return PA_OK;
}

const char* pa_status_string(pa_status status) {
    switch (status) {
        case PA_OK: return "PA_OK";
        case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG";
        case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED";
        case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE";
        case PA_ERR_CUDA: return "PA_ERR_CUDA";
        default: return "PA_UNKNOWN_STATUS";
    }
}

}  // extern "C"

// ----------------------------------------------------------------------------
// Split-K decode with library-owned scratch (no allocation by the caller or
// the library).  Some callers cannot allocate device memory when they launch
// work: plugins of inference runtimes that are handed only their inputs and
// outputs at enqueue time, or latency-critical loops where cudaMalloc's
// implicit device synchronisation would stall other streams.  For them, the
// fp32 partial results live in one fixed array in the library's device image.

namespace {

// The array is part of the module, so every GPU that loads the library holds
// it until the process exits.
constexpr size_t kStaticScratchBytes = PA_SPLITK_STATIC_SCRATCH_BYTES;
static __device__ __align__(256) float g_splitk_scratch[kStaticScratchBytes / sizeof(float)];

// Device address of g_splitk_scratch on the current device.  In host code
// the name g_splitk_scratch is only a host-side stand-in, so the address is
// looked up once per device (with that device current) and cached.
// A failed runtime call leaves its error as the thread's last error; it is
// cleared here so that a later launch check does not report it for an
// unrelated call.
pa_status static_scratch_address(void** ptr) {
    static std::mutex mu;
    static std::map<int, void*> cached;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    std::lock_guard<std::mutex> lock(mu);
    auto it = cached.find(dev);
    if (it == cached.end()) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_splitk_scratch) != cudaSuccess || p == nullptr) {
            cudaGetLastError();
            return PA_ERR_CUDA;
        }
        it = cached.emplace(dev, p).first;
    }
    *ptr = it->second;
    return PA_OK;
}

}  // namespace

extern "C" pa_status pa_decode_splitk_static(void* out, const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* block_tables, const int32_t* context_lens, float scale,
                                             int block_size, int num_seqs, int num_q_heads, int num_kv_heads,
                                             int head_dim, int max_blocks_per_seq, int max_context_len,
                                             int64_t num_blocks, pa_dtype dtype, int partition_size,
                                             void* stream) {
    // Requests whose partials do not fit the fixed array are refused before
    // any device work.
    size_t need = 0;
    const pa_status size_status =
        pa_decode_splitk_workspace_size(num_seqs, num_q_heads, head_dim, max_context_len, partition_size, &need);
    if (size_status != PA_OK) return size_status;
    if (need > kStaticScratchBytes) return PA_ERR_WORKSPACE;
    void* scratch = nullptr;
    const pa_status addr_status = static_scratch_address(&scratch);
    if (addr_status != PA_OK) return addr_status;
    // Two-launch form (no arrival counters): the partition kernel writes every
    // partial that the merge kernel reads (a partition whose copies timed out
    // is written as empty), so no part of the array has to start at zero and
    // the previous call's leftovers are never read.
    return pa_decode_splitk(out, q, k_cache, v_cache, block_tables, context_lens, scale, block_size, num_seqs,
                            num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, max_context_len, num_blocks,
                            dtype, partition_size, scratch, kStaticScratchBytes, nullptr, 0, nullptr, stream);
}

#ifdef PA_TEST_HOOKS
// ----------------------------------------------------------------------------
// Test hooks (libpa_test.so only; declared in pa_test.h).

namespace {

// One warp waits on an mbarrier that no thread or copy ever completes.
__global__ void pa_test_wait_kernel(unsigned long long limit_ns, long long* elapsed_ns) {
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x == 0) {
        pa::mbar_init(&bar, 1);
        pa::fence_barrier_init();
    }
    __syncwarp();
    const uint64_t t0 = pa::global_timer_ns();
    const bool done = pa::mbar_wait_bounded(&bar, 0, limit_ns);
    const uint64_t t1 = pa::global_timer_ns();
    if (threadIdx.x == 0) {
        if (!done) pa::flag_error(PA_DEVERR_TIMEOUT);
        *elapsed_ns = static_cast<long long>(t1 - t0);
    }
}

}  // namespace

// The hooks of the other translation unit (pa_ops.cu).
extern "C" __attribute__((visibility("hidden"))) cudaError_t pa_ops_set_hooks(unsigned long long limit_ns,
                                                                             int skip_first_copy);

extern "C" pa_status pa_test_set_hooks(int64_t wait_limit_ns, int skip_first_copy) {
    if (wait_limit_ns <= 0) return PA_ERR_INVALID_ARG;
    const unsigned long long limit = static_cast<unsigned long long>(wait_limit_ns);
    if (cudaMemcpyToSymbol(pa::g_test_wait_limit_ns, &limit, sizeof(limit)) != cudaSuccess) return PA_ERR_CUDA;
    if (cudaMemcpyToSymbol(pa::g_test_skip_first_copy, &skip_first_copy, sizeof(int)) != cudaSuccess)
        return PA_ERR_CUDA;
    return pa_ops_set_hooks(limit, skip_first_copy) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status pa_test_wait_timeout(int64_t limit_ns, int64_t* elapsed_ns, void* stream) {
    if (limit_ns <= 0 || !elapsed_ns || (reinterpret_cast<uintptr_t>(elapsed_ns) & 7u)) return PA_ERR_INVALID_ARG;
    pa_test_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<unsigned long long>(limit_ns),
                                                                         reinterpret_cast<long long*>(elapsed_ns));
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
#endif  // PA_TEST_HOOKS
