// What the library's two translation units share on the host: argument
// validation, kernel-variant dispatch on (dtype, head_dim, block_size) and the
// launches of the decode and prefill kernels.  pa_api.cu holds the entry points
// of pa.h, pa_ops.cu those of pa/ops.h; each compiles the kernel variants that
// its own entry points launch.
// Nothing here allocates device memory or synchronises.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <utility>
#include <map>
#include <mutex>
#include <tuple>

#include "pa.h"
#include "pa_decode.cuh"
#include "pa_prefill.cuh"
#include "pa_prefill_tc.cuh"

// Two CTA shapes for the decode kernels, measured on B200 over the benchmark
// workloads (warps per CTA, shared-memory ring bytes per warp):
//  * deep: one large CTA per SM with a two-stage ring per warp; best when the
//    grid is at most PA_DEEP_MAX_CTAS_PER_SM CTAs per SM (few, long
//    sequences per SM), where each CTA streams long enough to amortise its
//    start-up;
//  * wide: small CTAs, several resident per SM, so one CTA's start-up
//    (block-table read, first copies) and final merge overlap other CTAs'
//    streaming; best for grids of many short CTAs (split-K partitions,
//    batches of short sequences).
// (12 warps: with the launches made early, the Llama-3-8B step 48.0 -> 46.9
// us against 8 warps; 10 and 11 warps lie between)
#ifndef PA_DEEP_WARPS
#define PA_DEEP_WARPS 12
#endif
#ifndef PA_DEEP_RING
#define PA_DEEP_RING 16384
#endif
#ifndef PA_WIDE_WARPS
#define PA_WIDE_WARPS 4
#endif
#ifndef PA_WIDE_RING
#define PA_WIDE_RING 12288
#endif
// The same two shapes for 8-bit pools, whose blocks carry half the bytes
// for the same tensor-core work per block.
// (12 warps: with the launches made early, the Llama-3-8B decode over 8-bit pools
// 39.8 -> 38.9 us against 16 warps, the appending step 40.2 -> 40.1 us)
#ifndef PA_FP8_DEEP_WARPS
#define PA_FP8_DEEP_WARPS 12
#endif
#ifndef PA_FP8_DEEP_RING
#define PA_FP8_DEEP_RING 12288
#endif
#ifndef PA_FP8_WIDE_WARPS
#define PA_FP8_WIDE_WARPS 4
#endif
#ifndef PA_FP8_WIDE_RING
#define PA_FP8_WIDE_RING 8192
#endif
// Shared-prefix decode: the decode pass overlaps the prefix pass (1), or
// starts after it (0).  The prefix pass takes about this many CTAs (0: a
// third of the SMs; the decode pass fills the rest meanwhile): on the
// 128-sequence, 1024-token-prefix workload 48 of 148 (3 key partitions) ran
// 38.2 us, 32 39.4, 16 55.5, 64 41.3 and 148 51.3.
#ifndef PA_PREFIX_OVERLAP
#define PA_PREFIX_OVERLAP 1
#endif
// Launches may become resident before the work ahead of them ends (1), or
// not (0).  On steps launched back to back: Llama-3-8B decode 49.2 -> 47.4 us,
// the mix at 16-token blocks 38.0 -> 36.2 us, the shared-prefix step 37.4 ->
// 35.4 us, a step through the device block manager (three launches) 63.1 ->
// 57.2 us.
#ifndef PA_EARLY_LAUNCH
#define PA_EARLY_LAUNCH 1
#endif
#ifndef PA_PREFIX_CTAS
#define PA_PREFIX_CTAS 0
#endif
// ... and the decode pass's wide grid starts the sequences whose own part is
// in the upper (8 - N) / 8 of its range first (0: one class; 4 ran 40.3 us
// there against 47.3 us for one class).
#ifndef PA_PREFIX_CLASS_EIGHTHS
#define PA_PREFIX_CLASS_EIGHTHS 4
#endif

#ifndef PA_TWO_CLASS
#define PA_TWO_CLASS 1
#endif
#ifndef PA_DEEP_MAX_CTAS_PER_SM
#define PA_DEEP_MAX_CTAS_PER_SM 4
#endif

namespace {

enum class Kind { kDeep, kWide };

template <Kind K, bool FP8>
struct KindTuning;
// kRingCap bounds the K/V ring of a CTA.
template <>
struct KindTuning<Kind::kDeep, false> {
    static constexpr int kWarps = PA_DEEP_WARPS, kRing = PA_DEEP_RING, kRingCap = 200 * 1024;
};
template <>
struct KindTuning<Kind::kWide, false> {
    static constexpr int kWarps = PA_WIDE_WARPS, kRing = PA_WIDE_RING, kRingCap = 200 * 1024;
};
template <>
struct KindTuning<Kind::kDeep, true> {
    static constexpr int kWarps = PA_FP8_DEEP_WARPS, kRing = PA_FP8_DEEP_RING, kRingCap = 200 * 1024;
};
template <>
struct KindTuning<Kind::kWide, true> {
    static constexpr int kWarps = PA_FP8_WIDE_WARPS, kRing = PA_FP8_WIDE_RING, kRingCap = 200 * 1024;
};


// 16-bit pools of 32-token blocks take wide CTAs of this many warps (one 16
// KiB stage each): on the continuous-batching mix two warps per CTA with the
// long sequences started first ran 40.1 us, four warps 41.7 us (and 43.2 with
// the long sequences first), three 41.2, one 54.4.
#ifndef PA_WIDE32_WARPS
#define PA_WIDE32_WARPS 2
#endif

// FP8: the pools hold 1-byte e4m3 codes, so a stage is half the size of a
// 16-bit one and the same ring bytes hold twice the stages.
template <typename T, int D, int B, Kind K, bool FP8 = false>
struct DecodeConfig {
    static constexpr int kElem = FP8 ? 1 : static_cast<int>(sizeof(T));
    static constexpr int kStageBytes = 2 * B * D * kElem;                       // K + V tile
    static constexpr int kRingCap = KindTuning<K, FP8>::kRingCap;                    // ring bytes per CTA at most
    static constexpr int kMaxWarps = kRingCap / kStageBytes;
    static constexpr int kWarpsWanted =
        (K == Kind::kWide && !FP8 && B == 32 && sizeof(T) == 2) ? PA_WIDE32_WARPS : KindTuning<K, FP8>::kWarps;
    static constexpr int kWarps = kWarpsWanted < kMaxWarps ? kWarpsWanted : kMaxWarps;
    static constexpr int kRaw = KindTuning<K, FP8>::kRing / kStageBytes;
    static constexpr int kFit = kRingCap / (kWarps * kStageBytes);
    static constexpr int kStages0 = kRaw < 1 ? 1 : (kRaw > 16 ? 16 : kRaw);
    static constexpr int kStages = kStages0 < kFit ? kStages0 : kFit;
    using Smem = pa::DecodeSmem<T, D, B, kWarps, kStages, FP8>;
    static_assert(kStages >= 1, "one stage per warp at least");
    static_assert(Smem::kTotal <= 227 * 1024, "shared memory per CTA");
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int elem_size(pa_dtype dt) { return dt == PA_F32 ? 4 : 2; }

bool dtype_ok(int dt) { return dt == PA_F32 || dt == PA_F16 || dt == PA_BF16; }

// Raises the dynamic shared-memory limit of `kernel` on the current device to
// the device's opt-in maximum, once per (kernel, device).  Setting it to the
// largest value (rather than to one launch's size) keeps every later launch
// of any size within the limit.
cudaError_t ensure_smem(const void* kernel) {
    static std::mutex mu;
    static std::map<std::pair<const void*, int>, bool> done;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count({kernel, dev})) return cudaSuccess;
    int optin = 0;
    e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes attr{};
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             optin - static_cast<int>(attr.sharedSizeBytes));
    if (e == cudaSuccess) done[{kernel, dev}] = true;
    return e;
}

// Every launch is a programmatic dependent launch (each kernel first waits
// for the work ahead of it on the stream, see wait_for_prior_work): a grid
// may take its places on the SMs before that work ends, which hides the
// launch latency between the library's launches.
template <typename... KArgs, typename... Args>
cudaError_t launch_early(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                         int early, Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = early;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename T>
struct TypeTag {
    using type = T;
};
template <int V>
struct IntTag {
    static constexpr int value = V;
};

// Calls f(TypeTag<T>, IntTag<D>, IntTag<B>) for the kernel variant of
// (dtype, head_dim, block_size); the shape has been validated already.
template <typename F>
cudaError_t with_variant(pa_dtype dt, int D, int B, F&& f) {
    auto by_block = [&](auto tt, auto dd) -> cudaError_t {
        switch (B) {
            case 8: return f(tt, dd, IntTag<8>{});
            case 16: return f(tt, dd, IntTag<16>{});
            case 32: return f(tt, dd, IntTag<32>{});
            default: return cudaErrorInvalidValue;
        }
    };
    auto by_dim = [&](auto tt) -> cudaError_t {
        switch (D) {
            case 64: return by_block(tt, IntTag<64>{});
            case 128: return by_block(tt, IntTag<128>{});
            default: return cudaErrorInvalidValue;
        }
    };
    switch (dt) {
        case PA_F32: return by_dim(TypeTag<float>{});
        case PA_F16: return by_dim(TypeTag<__half>{});
        case PA_BF16: return by_dim(TypeTag<__nv_bfloat16>{});
        default: return cudaErrorInvalidValue;
    }
}

template <typename T, int D, int B, bool SPLIT, Kind K, bool FP8 = false, bool PREFIX = false, bool WINDOW = false>
cudaError_t launch_decode(const pa::DecodeParams& p, dim3 grid, cudaStream_t stream) {
    using C = DecodeConfig<T, D, B, K, FP8>;
    auto kernel = pa::pa_decode_kernel<T, D, B, C::kWarps, C::kStages, SPLIT, FP8,
                                       !SPLIT && (!PREFIX || PA_PREFIX_CLASS_EIGHTHS > 0) && K == Kind::kWide,
                                       PREFIX, WINDOW>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
    // The shared-prefix form's CTAs start while the prefix pass (the launch
    // before, on the same stream) still runs: the two grids meet only through
    // the arrival counters, and one CTA waits for the prefix pass to complete
    // (so that this grid ends after it).
    return launch_early(kernel, grid, dim3(C::kWarps * 32), C::Smem::kTotal, stream,
                        PREFIX ? PA_PREFIX_OVERLAP : PA_EARLY_LAUNCH, p);
}

// Streaming multiprocessors of the current device, once per device.
int sm_count() {
    static std::mutex mu;
    static std::map<int, int> counts;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    auto it = counts.find(dev);
    if (it != counts.end()) return it->second;
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return counts[dev] = n;
}

// The split kernel always runs wide CTAs; the one-pass kernel runs deep CTAs
// unless its grid holds more than PA_DEEP_MAX_CTAS_PER_SM CTAs per SM.
template <bool SPLIT, bool FP8 = false, bool PREFIX = false, bool WINDOW = false>
cudaError_t decode_dispatch(pa_dtype dt, int D, int B, const pa::DecodeParams& p, dim3 grid, cudaStream_t st) {
    const long long ctas = static_cast<long long>(grid.x) * grid.y * grid.z;
    // (partitions of a window: deep where the SMs hold them all at once)
    const bool deep = SPLIT ? WINDOW && ctas <= sm_count()
                            : ctas <= static_cast<long long>(PA_DEEP_MAX_CTAS_PER_SM) * sm_count();
    return with_variant(dt, D, B, [&](auto tt, auto dd, auto bb) -> cudaError_t {
        using T = typename decltype(tt)::type;
        constexpr int kD = decltype(dd)::value, kB = decltype(bb)::value;
        if constexpr ((FP8 || PREFIX) && pa::IsF32<T>::value) {
            return cudaErrorInvalidValue;  // 16-bit only (refused on the host first)
        } else if constexpr (PREFIX) {
            return deep ? launch_decode<T, kD, kB, false, Kind::kDeep, false, true>(p, grid, st)
                        : launch_decode<T, kD, kB, false, Kind::kWide, false, true>(p, grid, st);
        } else if constexpr (SPLIT) {
            if constexpr (WINDOW)
                if (deep) return launch_decode<T, kD, kB, true, Kind::kDeep, FP8, false, true>(p, grid, st);
            return launch_decode<T, kD, kB, true, Kind::kWide, FP8, false, WINDOW>(p, grid, st);
        } else {
            return deep ? launch_decode<T, kD, kB, false, Kind::kDeep, FP8, false, WINDOW>(p, grid, st)
                        : launch_decode<T, kD, kB, false, Kind::kWide, FP8, false, WINDOW>(p, grid, st);
        }
    });
}

// A one-pass launch of many small CTAs (the wide shape) without a start
// order from the host starts the long sequences first by running the grid
// twice over: the first half takes the sequences of at least a quarter of
// max_context_len tokens, the second half the others (CTAs start roughly in
// blockIdx order; a CTA of the other class leaves at once).
dim3 two_class_grid(pa::DecodeParams& p, dim3 grid, int max_context_len, int block_size, int threshold = -1) {
    const long long ctas = static_cast<long long>(grid.x) * grid.y * grid.z;
    const bool wide = ctas > static_cast<long long>(PA_DEEP_MAX_CTAS_PER_SM) * sm_count();
    if (threshold < 0) threshold = PA_TWO_CLASS && max_context_len >= 4 ? max_context_len / 4 : 0;
    if (threshold <= 0 || !wide || p.seq_order != nullptr || 2LL * grid.z > 65535)
        return grid;
    p.class_threshold = threshold;
    grid.z *= 2;
    return grid;
}

template <typename T, int D>
cudaError_t launch_merge(const pa::MergeParams& p, cudaStream_t st) {
    constexpr bool kLog2 = !pa::IsF32<T>::value;
    const long long warps = static_cast<long long>(p.num_seqs) * p.num_q_heads;
    const unsigned blocks = static_cast<unsigned>((warps + 3) / 4);
    return launch_early(pa::pa_merge_kernel<T, D, kLog2>, dim3(blocks), dim3(128), 0, st, PA_EARLY_LAUNCH, p);
}

cudaError_t merge_dispatch(pa_dtype dt, int D, const pa::MergeParams& p, cudaStream_t st) {
    if (D == 64) {
        if (dt == PA_F32) return launch_merge<float, 64>(p, st);
        if (dt == PA_F16) return launch_merge<__half, 64>(p, st);
        return launch_merge<__nv_bfloat16, 64>(p, st);
    }
    if (dt == PA_F32) return launch_merge<float, 128>(p, st);
    if (dt == PA_F16) return launch_merge<__half, 128>(p, st);
    return launch_merge<__nv_bfloat16, 128>(p, st);
}

struct DecodeShape {
    int block_size, num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, max_context_len;
    long long num_blocks;
    int dtype;
};

pa_status check_decode(const void* out, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, const int32_t* context_lens, float scale,
                       const DecodeShape& sh) {
    if (sh.num_seqs < 0 || sh.num_q_heads <= 0 || sh.num_kv_heads <= 0 || sh.head_dim <= 0 ||
        sh.block_size <= 0 || sh.max_blocks_per_seq < 0 || sh.max_context_len < 0 || sh.num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    if (!dtype_ok(sh.dtype)) return PA_ERR_UNSUPPORTED;
    if (sh.head_dim != 64 && sh.head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (sh.block_size != 8 && sh.block_size != 16 && sh.block_size != 32) return PA_ERR_UNSUPPORTED;
    if (sh.num_q_heads % sh.num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    const int g = sh.num_q_heads / sh.num_kv_heads;
    if (g != 1 && g != 2 && g != 4 && g != 8) return PA_ERR_UNSUPPORTED;
    if (sh.num_seqs > 65535 || sh.num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;  // grid limits
    if (sh.num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned4(block_tables) || !aligned4(context_lens))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

int context_cap(const DecodeShape& sh) {
    const long long by_table = static_cast<long long>(sh.max_blocks_per_seq) * sh.block_size;
    const long long cap = by_table < sh.max_context_len ? by_table : sh.max_context_len;
    return cap > INT_MAX ? INT_MAX : static_cast<int>(cap);
}

pa::DecodeParams make_params(void* out, const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, const int32_t* context_lens, float scale,
                             const DecodeShape& sh) {
    pa::DecodeParams p{};
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    // 16-bit path keeps scores in base 2: fold log2(e) into the scale.
    p.score_scale = sh.dtype == PA_F32 ? scale : scale * 1.4426950408889634f;
    p.num_seqs = sh.num_seqs;
    p.num_q_heads = sh.num_q_heads;
    p.num_kv_heads = sh.num_kv_heads;
    p.group = sh.num_q_heads / sh.num_kv_heads;
    p.max_blocks_per_seq = sh.max_blocks_per_seq;
    p.context_cap = context_cap(sh);
    p.num_blocks = sh.num_blocks;
    return p;
}

size_t splitk_bytes(long long seqs, long long heads, long long parts, long long head_dim) {
    return static_cast<size_t>(seqs * heads * parts * (head_dim + 2) * 4);
}

// 64-key tiles of a shared prefix of prefix_blocks blocks: the most key
// partitions the prefix pass can take.
int shared_prefix_tiles(int prefix_blocks, int block_size) {
    return static_cast<int>((static_cast<long long>(prefix_blocks) * block_size + 63) / 64);
}

// Device memory, or page-locked host memory mapped into the device's address
// space (what the copy kernel can dereference).
bool device_accessible(const void* p) {
    cudaPointerAttributes attr{};
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();  // the failed query leaves an error behind; clear it
        return false;
    }
    if (attr.type == cudaMemoryTypeDevice || attr.type == cudaMemoryTypeManaged) return true;
    return attr.type == cudaMemoryTypeHost && attr.devicePointer == p;
}

// Chunked prefill: 4 warps (64 MMA rows) per CTA, a 4-stage block ring.
constexpr int kPrefillWarps = 4;
constexpr int kPrefillStages = 4;

// Blocks of 8, 16 or 32 tokens run the 5th-generation tensor-core kernel (two
// query tiles of 128 MMA rows per CTA); PA_PREFILL_TC=0 or a K pool that no
// tensor map can describe run the warp-level one.
#ifndef PA_PREFILL_TC
#define PA_PREFILL_TC 1
#endif

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime
// (the library links no driver library); null where there is no driver.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// The K pool viewed as a 2-D tensor of rows (block, kv head, 8-dim chunk), each
// row the chunk's B tokens x 8 elements (B * 16 bytes), one row per box: the
// operand of the prefill kernel's gather4 loads.  False when it cannot be
// described (no driver, or more rows than a 32-bit coordinate reaches).
bool encode_k_rows(CUtensorMap* map, const void* k_cache, pa_dtype dt, int B, int D, int Hkv, long long num_blocks) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return false;
    const long long rows = num_blocks * Hkv * (D / 8);
    if (rows <= 0 || rows > INT_MAX) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(B) * 8, static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(B) * 16};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(B) * 8, 1};
    const cuuint32_t elem_strides[2] = {1, 1};
    const CUtensorMapDataType type =
        dt == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return encode(map, type, 2, const_cast<void*>(k_cache), dims, strides, box, elem_strides,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tensor-core kernel's K operand: blocks of 8 tokens are bulk-copied
// whole and need no tensor map; larger blocks are gathered through one.
bool prefill_k_source(CUtensorMap* map, const void* k_cache, pa_dtype dt, int B, int D, int Hkv,
                      long long num_blocks) {
    return B == 8 || encode_k_rows(map, k_cache, dt, B, D, Hkv, num_blocks);
}

// Query tiles (of 128 MMA rows) per tensor-core prefill CTA: 2 (one CTA per
// SM, the two tiles sharing every K/V tile) or 1 (two CTAs per SM, each with
// its own K/V stream).  On the chunked-prefill workload one tile per CTA ran
// 197.4 against 208.6 us at 32-token blocks, but 228.0 against 221.1 at 16 and
// 273.2 against 236.6 at 8 (twice the copies per SM), and the shared-prefix
// step 44.3 against 36.1 us; so 32-token blocks take one (PA_PF_QT32).
#ifndef PA_PF_QT32
#define PA_PF_QT32 1
#endif
constexpr int prefill_tiles_per_cta(int block_size, bool prefix) {
    return (block_size == 32 && !prefix) ? PA_PF_QT32 : 2;
}

template <typename T, int D, int B, bool PREFIX = false, bool WINDOW = false>
cudaError_t launch_prefill_tc(const pa::PrefillParams& p, const CUtensorMap& k_rows, dim3 grid, cudaStream_t st) {
    constexpr int kQT = prefill_tiles_per_cta(B, PREFIX);
    using Sm = pa::PrefillTcSmem<T, D, B, kQT>;
    auto kernel = pa::pa_prefill_tc_kernel<T, D, B, PREFIX, kQT, WINDOW>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
    return launch_early(kernel, grid, dim3((6 * kQT + 2) * 32), Sm::kTotal, st, PA_EARLY_LAUNCH, p, k_rows);
}

template <typename T, int D, int B>
cudaError_t launch_prefill(const pa::PrefillParams& p, dim3 grid, cudaStream_t st) {
    using Sm = pa::PrefillSmem<T, D, B, kPrefillWarps, kPrefillStages>;
    auto kernel = pa::pa_prefill_kernel<T, D, B, kPrefillWarps, kPrefillStages>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
    return launch_early(kernel, grid, dim3(kPrefillWarps * 32), Sm::kTotal, st, PA_EARLY_LAUNCH, p);
}

// The one-pass and split decode bodies, shared by the 16-bit-pool entries
// (FP8 = false) and the 8-bit-pool entries (FP8 = true, with K/V scales).
template <bool FP8>
pa_status check_scales(const DecodeShape& sh, const float* k_scale, const float* v_scale) {
    if constexpr (FP8) {
        if (sh.dtype == PA_F32) return PA_ERR_UNSUPPORTED;  // 8-bit pools take 16-bit queries
        if (sh.num_seqs > 0 && (!k_scale || !v_scale || !aligned4(k_scale) || !aligned4(v_scale)))
            return PA_ERR_INVALID_ARG;
    }
    return PA_OK;
}

template <bool FP8>
pa_status decode_one_pass(void* out, const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                          const float* v_scale, const int32_t* block_tables, const int32_t* context_lens,
                          float scale, const DecodeShape& sh, const int32_t* seq_order, void* stream,
                          const void* new_key = nullptr, const void* new_value = nullptr,
                          const int32_t* ref_counts = nullptr) {
    pa_status st = check_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    if (st == PA_OK) st = check_scales<FP8>(sh, k_scale, v_scale);
    if (st != PA_OK || sh.num_seqs == 0) return st;
    if (!aligned4(seq_order)) return PA_ERR_INVALID_ARG;
    pa::DecodeParams p = make_params(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    p.seq_order = seq_order;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.new_key = new_key;
    p.new_value = new_value;
    p.ref_counts = ref_counts;
    const dim3 grid = two_class_grid(p, dim3(1, sh.num_kv_heads, sh.num_seqs), sh.max_context_len, sh.block_size);
    const cudaError_t e = decode_dispatch<false, FP8>(static_cast<pa_dtype>(sh.dtype), sh.head_dim, sh.block_size,
                                                      p, grid, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <bool FP8>
pa_status decode_split(void* out, const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                       const float* v_scale, const int32_t* block_tables, const int32_t* context_lens, float scale,
                       const DecodeShape& sh, int partition_size, void* workspace, size_t workspace_bytes,
                       int32_t* counters, int64_t num_counters, const int32_t* seq_order, void* stream) {
    pa_status st = check_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    if (st == PA_OK) st = check_scales<FP8>(sh, k_scale, v_scale);
    if (st != PA_OK) return st;
    const int block_size = sh.block_size, num_seqs = sh.num_seqs, num_q_heads = sh.num_q_heads;
    const int num_kv_heads = sh.num_kv_heads, head_dim = sh.head_dim;
    const pa_dtype dtype = static_cast<pa_dtype>(sh.dtype);
    if (partition_size <= 0 || partition_size % 16 != 0 || partition_size % block_size != 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!aligned4(seq_order)) return PA_ERR_INVALID_ARG;
    pa::DecodeParams p = make_params(out, q, k_cache, v_cache, block_tables, context_lens, scale, sh);
    p.seq_order = seq_order;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    const int pb = partition_size / block_size;
    const long long cap_blocks = (static_cast<long long>(p.context_cap) + block_size - 1) / block_size;
    const long long parts = (cap_blocks + pb - 1) / pb;
    if (parts > INT_MAX) return PA_ERR_UNSUPPORTED;
    const size_t need = splitk_bytes(num_seqs, num_q_heads, parts, head_dim);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return PA_ERR_WORKSPACE;
    float* acc = static_cast<float*>(workspace);
    p.part_acc = acc;
    p.part_ml = acc + static_cast<size_t>(num_seqs) * num_q_heads * parts * head_dim;
    p.partition_blocks = pb;
    p.num_partitions = static_cast<int>(parts);
    if (counters != nullptr) {
        if (!aligned4(counters) || num_counters < static_cast<int64_t>(num_seqs) * num_kv_heads)
            return PA_ERR_WORKSPACE;
        p.counters = counters;
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (parts > 0) {
        const dim3 grid(static_cast<unsigned>(parts), num_kv_heads, num_seqs);
        const cudaError_t e = decode_dispatch<true, FP8>(dtype, head_dim, block_size, p, grid, s);
        if (e != cudaSuccess) return PA_ERR_CUDA;
        if (counters != nullptr) return PA_OK;  // merged inside the partition kernel
    }
    pa::MergeParams m{};
    m.out = out;
    m.part_acc = p.part_acc;
    m.part_ml = p.part_ml;
    m.context_lens = context_lens;
    m.num_seqs = num_seqs;
    m.num_q_heads = num_q_heads;
    m.context_cap = p.context_cap;
    m.block_size = block_size;
    m.partition_blocks = pb;
    m.num_partitions = static_cast<int>(parts);
    return merge_dispatch(dtype, head_dim, m, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
