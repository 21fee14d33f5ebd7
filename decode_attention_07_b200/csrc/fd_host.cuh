// fd_host.cuh -- what the library's translation units share on the host side:
// argument checks, workspace layout, tensor-map encoding (one cache per
// device), test hooks, and the split kernel's launch. Defined in fd_api.cu
// unless inline.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>
#include <mutex>

#include "fd.h"
#include "fd_split.cuh"

namespace fdh {

constexpr int kMaxDevices = 64;
constexpr float kLog2e = 1.4426950408889634f;

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [a, a + an) and [b, b + bn) share a byte.
inline bool overlap(const void *a, size_t an, const void *b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return an > 0 && bn > 0 && x < y + bn && y < x + an;
}

int check_shape(int B, int Hq, int Hkv, int D, int max_len);
size_t align256(size_t x);

// Workspace: seg_out [slots][g][D] fp32 | seg_lse [slots][g] fp32 | row tickets [B*Hkv] int32
// followed by chunk tickets [slots] int32,
// each part 256-byte aligned.
struct WorkspaceLayout {
    size_t seg_out, seg_lse, tickets, total;
};
WorkspaceLayout workspace_layout(int B, int Hq, int Hkv, int D, int num_splits);
size_t workspace_bytes(int B, int Hq, int Hkv, int D, int num_splits);

// Current device (FD_ERR_DEVICE if there is none), and its SM count once it
// is known to be one the library is built for.
int current_device(int *dev);
int device_sms(int *sms);

// Tensor maps (see the definitions).
int encode_cache_map(CUtensorMap *map, const void *base, int D, int Lmax, long long rows, bool one_byte = false);
int encode_cache_map_rows(CUtensorMap *map, const void *base, int Lmax, long long rows);
int encode_paged_map(CUtensorMap *map, const void *base, int D, int page_size, int Hkv, long long num_pages, bool nhd,
                     bool one_byte = false);
int encode_paged_run_map(CUtensorMap *map, const void *base, int D, int page_size, int Hkv, long long num_pages,
                         bool nhd, bool one_byte);

// Test hooks (see the definitions).
bool inject_launch_failure();
int debug_withhold();
int debug_spoil_guess();

struct Problem {
    int B, Hq, Hkv, D, max_len;
    const uint16_t *q, *k, *v;
    const int32_t *seqlens;
    float scale;
    float *out, *lse;
    void *ws;
    size_t ws_bytes;
    int num_splits;
    cudaStream_t stream;
};
Problem make_problem(int B, int Hq, int Hkv, int D, int max_len, const uint16_t *q, const uint16_t *k,
                     const uint16_t *v, const int32_t *seqlens, float scale, float *out, float *lse, void *ws,
                     size_t ws_bytes, int num_splits, void *stream);
int check_problem(const Problem &pr, bool need_kv);
void seg_pointers(const Problem &pr, float **so, float **sl, int **tickets, int q_len = 1);

struct PagedLayout {
    const int32_t *block_table;
    int page_size, num_pages, max_pages;
    bool nhd;
};
// Page size, pool size, block-table width and layout, and the length they
// give (no CUDA call): FD_OK or FD_ERR_SHAPE.
int check_paged(int page_size, int num_pages, int max_pages_per_seq, int kv_layout, long long *max_len);

// Tokens per scale block of an 8-bit cache: 16, 32, 64 or 128.
inline bool valid_block(int block_tokens) {
    return block_tokens >= 16 && block_tokens <= 128 && (block_tokens & (block_tokens - 1)) == 0;
}

// The split kernel's parameters for a problem over a contiguous cache
// (pl == nullptr) or a paged one. q_len > 1: several queries per sequence
// (pr.Hq counts query heads of one query position).
fd::SplitParams split_params(const Problem &pr, int q_len, const PagedLayout *pl);

// Reads and clears the error word of one translation unit's kernels on the
// current device (each unit that instantiates the split kernel has its own).
template <class Word>
int take_error_word(Word &symbol, int *word) {
    const int zero = 0;
    if (cudaMemcpyFromSymbol(word, symbol, sizeof *word) != cudaSuccess ||
        cudaMemcpyToSymbol(symbol, &zero, sizeof zero) != cudaSuccess) {
        cudaGetLastError();
        return FD_ERR_LAUNCH;
    }
    return FD_OK;
}
int take_block_error(int *word);     // fd_block.cu
int take_weights_error(int *word);   // fd_weights.cu

// ---------------------------------------------------------------- launches --
template <int D, class Consumer, bool kFused, bool kPaged>
int launch_split_t(const CUtensorMap &tk, const CUtensorMap &tv, const fd::SplitParams &p, cudaStream_t st,
                   const CUtensorMap *rk = nullptr, const CUtensorMap *rv = nullptr) {
    constexpr int smem = fd::SplitConfig<D, Consumer::G, Consumer::kElemBytes, kPaged>::kSmemBytes;
    auto kern = fd::fd_split_kernel<D, Consumer, kFused, kPaged>;
    // the attribute is per function and device; set it once per device
    static std::once_flag once[kMaxDevices];
    static cudaError_t attr_err[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return FD_ERR_DEVICE;
    }
    std::call_once(once[dev], [&] {
        attr_err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (attr_err[dev] != cudaSuccess) {
        cudaGetLastError();
        return FD_ERR_LAUNCH;
    }
    // programmatic dependent launch: the prologue overlaps the previous
    // kernel's tail; the kernel waits for it before reading any input
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(p.P));
    cfg.blockDim = dim3(fd::split_threads<kPaged>());
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (inject_launch_failure()) return FD_ERR_LAUNCH;
    // the maps of consecutive page runs (small pages only; never read otherwise)
    if (cudaLaunchKernelEx(&cfg, kern, tk, tv, rk ? *rk : tk, rv ? *rv : tv, p) != cudaSuccess) {
        cudaGetLastError();
        return FD_ERR_LAUNCH;
    }
    return FD_OK;
}

// One launch of `kern`, as a programmatic dependent of the previous kernel on
// the stream (kern waits for it before it reads anything).
template <class Kernel, class... Args>
int launch_dependent(Kernel kern, dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster, Args... args) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (inject_launch_failure()) return FD_ERR_LAUNCH;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
        cudaGetLastError();
        return FD_ERR_LAUNCH;
    }
    return FD_OK;
}

}  // namespace fdh
