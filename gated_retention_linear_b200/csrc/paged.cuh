// paged.cuh -- host interface of the paged key-value cache: decode attention over it
// (paged_attention.cu) and its upkeep (paged_cache.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "gret.h"

namespace gret {

constexpr int PAGED_MAX_PAGE = 1024;      // tokens a page; a power of two
constexpr int PAGED_MAX_SEQS = 16384;     // rows of a page table: the plan kernels keep 8 bytes of
                                          // each row in shared memory

// The pool: row (token slot t, head h) of page p is row_bytes bytes at k + p*sp + t*st + h*sh.
// All strides are in bytes here.
struct PagedPool {
    unsigned char* k;
    unsigned char* v;
    int64_t sp, st, sh;
    int n_pages;
    int page_shift;      // log2(page size)
    int H;               // heads of a slot
    int row_bytes;       // a multiple of 16
};

// The page table: entry j of row s at entries[s * stride + j], j < max_pages.
struct PagedTable {
    int32_t* entries;
    int64_t stride;
    int max_pages;
    int S;
};

struct PagedAttnArgs {
    const void* q;           // [B, Hq, d]
    const int32_t* seq_lens; // [B]
    PagedTable table;        // S = B
    PagedPool pool;          // H = Hkv
    bool bf16;
    float scale;
    int window;              // 0: no window
    int Hq, d;
    void* o;                 // [B, Hq, d]
    float* lse;              // [B, Hq] or nullptr
    int32_t* status;         // or nullptr
    void* workspace;
};

size_t paged_attn_workspace(bool bf16, int Hq, int Hkv, int d);
cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream);

struct PagedAppendArgs {
    const unsigned char* k;  // token i, head h at k + i*kt + h*kh (bytes)
    const unsigned char* v;
    int64_t kt, kh, vt, vh;
    int64_t T;
    const int32_t* cu_seqlens;  // [S + 1] or nullptr (token i belongs to row i)
    const int32_t* pos;         // [S]
    PagedTable table;
    PagedPool pool;
    int32_t* status;
};

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream);

struct PagedResizeArgs {
    const int32_t* delta;    // [S]
    int32_t* seq_lens;       // [S]
    int32_t* pos;            // [S]
    int32_t* ref;            // [n_pages]
    PagedTable table;
    PagedPool pool;
    int32_t* status;
    int32_t* workspace;      // [S]
};

cudaError_t launch_paged_resize(const PagedResizeArgs& a, cudaStream_t stream);

struct PagedForkArgs {
    const int32_t* src;      // [n]
    const int32_t* dst;      // [n]
    int n;
    int32_t* seq_lens;       // [S]
    int32_t* ref;            // [n_pages]
    PagedTable table;
    int n_pages, page_shift;
    int32_t* status;
};

cudaError_t launch_paged_fork(const PagedForkArgs& a, cudaStream_t stream);

struct PagedCompactArgs {
    const int32_t* seq_lens; // [S]
    int32_t* ref;            // [n_pages]
    int32_t* n_live;         // [1]
    PagedTable table;
    PagedPool pool;
    int32_t* status;
    int32_t* workspace;      // 4 + 3 * n_pages
};

cudaError_t launch_paged_compact(const PagedCompactArgs& a, cudaStream_t stream);

}  // namespace gret

#ifdef __CUDACC__
namespace gret {

// The kernels of the paged cache are launched so that they may start while the one before them in
// the stream ends (programmatic dependent launch): a kernel's blocks are in place when that one is
// done, which saves a microsecond or so a launch.  Each waits for that end itself, every block of
// it, so that its own end means the end of all before it: wait_for_previous(), before the first
// access to memory that others write.  Only then does a kernel let its successor start.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                         cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Dynamic shared memory of `bytes`, at most `most`, for a kernel: up to 24 KB beside its own arrays
// need no leave; for more it is asked once on each of the first 64 devices.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes, int most) {
    static std::atomic<uint64_t> given{0};
    if (bytes <= 24 * 1024) return cudaSuccess;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
    if (given.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) given.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void paged_flag(int32_t* status, int bit) {
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ int pages_of(int64_t n, int page_shift) {
    return (int)((n + (1 << page_shift) - 1) >> page_shift);
}

}  // namespace gret
#endif
