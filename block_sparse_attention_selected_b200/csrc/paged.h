// paged.h -- internal launch interface of the paged K/V cache (paged.cu, paged_attn.cu,
// paged_few.cu, paged_api.cu), and the host helpers it shares with api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <mutex>
#include <utility>

#include "../../include/nsa_sel.h"
#include "nsa_common.cuh"

namespace nsa {

// Programmatic dependent launch: the kernels of a step follow one another within
// microseconds, so each is launched while the one before it still runs, sets itself up, and
// waits for the end of everything before it (depend()) before it touches memory; it lets the
// next one do the same from its own start (release_dependents()).  What such a kernel reads may
// be written while it is already running, so none of its loads takes the read-only path (__ldg).
__device__ __forceinline__ void depend() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void release_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             A&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// Host helpers of the C ABI (api.cu).
nsa_status_t check_device(int* num_sms, nsa_stream_t stream);
PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn();   // null if the driver lacks it
// The kernels of one call hand their results over through its workspace.  Threads that share a
// stream and a workspace (the binding keeps one per stream) therefore launch whole calls, one
// after the other: held from a call's first launch to its last.
class LaunchLock {
public:
    explicit LaunchLock(const void* workspace);

private:
    std::lock_guard<std::mutex> lock_;
};

// The paged-attention kernels report one status byte per CTA, in the unused end of the status
// block (every other call clears the whole block first).
constexpr int kMaxStatusCtas = 160;
static_assert(sizeof(DevStatus::pad) >= kMaxStatusCtas, "one status byte per CTA");
__host__ __device__ inline unsigned char* cta_status(DevStatus* st) {
    return reinterpret_cast<unsigned char*>(st->pad);
}

struct PagedPlanArgs {
    const int32_t* new_lens; // [R]
    const int32_t* old_lens; // [R]
    int R;
    const int32_t* free_pages;
    int num_free;
    int32_t* table;          // [R, width], row stride table_stride
    int width;
    long long table_stride;
    int ps;                  // tokens per page
    int T;                   // rows of slots and positions
    int32_t* cu;             // [R + 1]
    int32_t* kv_lens;        // [R]
    int64_t* slots;          // [T]
    int32_t* positions;      // [T]
    int32_t* pages_used;     // [1]
};
cudaError_t launch_paged_plan(const PagedPlanArgs& p, int num_sms, cudaStream_t stream);

// Strides in elements of 16 bits.
struct PagedWriteArgs {
    const uint16_t* k;
    const uint16_t* v;
    long long k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    const int64_t* slots;    // [T]
    int T, hkv, d;
    uint16_t* k_cache;
    uint16_t* v_cache;
    int num_pages, ps;
    long long page_stride, token_stride, head_stride;
};
cudaError_t launch_paged_write(const PagedWriteArgs& p, cudaStream_t stream);

struct PagedAttnArgs {
    const uint16_t* q;       // [T, hq, d]
    long long q_token_stride, q_head_stride;
    const uint16_t* k;       // the caches
    const uint16_t* v;
    long long page_stride, token_stride, head_stride;
    int num_pages, ps;
    int T, R, hq, hkv, G, d;
    const int32_t* cu;       // [R + 1] new tokens
    const int32_t* kv_lens;  // [R] tokens in the cache, the new ones included
    const int32_t* table;    // [R, table_width]
    int table_width;
    long long table_stride;
    const int32_t* bidx;     // [T, hkv, topk] or null: every visible key
    int topk, bs;
    int swin;                // sliding window in keys (0: none)
    float scale_log2;        // scale * log2(e)
    uint16_t* out;           // [T, hq, d]
    float* lse;              // [hq, T] or null
    DevStatus* st;
    bool test_skip;          // NSA_TEST_SKIP_ARRIVE: the first K tile of CTA 0 never counts as there
};
size_t paged_attn_workspace(int d);   // bytes, the status block included
cudaError_t launch_paged_attn(const PagedAttnArgs& p, int f16, int num_sms, cudaStream_t stream);

}  // namespace nsa
