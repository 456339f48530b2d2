// paged.cu -- the bookkeeping of a paged K/V cache: block tables and slot maps from
// request lengths, and the write of new K/V rows into their slots.
//
// A request r holds old_r tokens in its cache and brings new_r more.  With pages of ps
// tokens it holds have_r = ceil(old_r / ps) pages and needs need_r = ceil((old_r +
// new_r) / ps); its need_r - have_r fresh pages are taken from the free list in request
// order, so that their places in it are exclusive prefix sums over the requests.
#include <algorithm>

#include "paged.h"

namespace nsa {
namespace {

constexpr int kPlanThreads = 512;

__device__ __forceinline__ int saturate(long long x) {
    return (int)(x < 0x7fffffffLL ? x : 0x7fffffffLL);
}

// One launch, no pass between blocks: every block scans the request lengths by itself
// (two int32 reads per request, from L2) into shared memory, then takes its stripe of
// the fresh pages and of the tokens.  Bound by latency: 3.4 us for 64 requests of one token,
// 7.1 us for 1000 requests with 130,000 tokens (12 bytes out per token).  A token's slot on a
// fresh page comes from the free list and not from the table entry that another block may be
// writing.
__global__ void __launch_bounds__(kPlanThreads) k_paged_plan(PagedPlanArgs p) {
    extern __shared__ int plan_smem[];
    int* cu = plan_smem;                    // [R + 1] tokens before request r
    int* pre = plan_smem + p.R + 1;         // [R + 1] fresh pages before request r
    __shared__ long long wsum[2][kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    release_dependents();
    depend();
    const int per = (p.R + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
    auto pages = [&](long long tokens) -> int {
        return (int)min((tokens + p.ps - 1) / p.ps, (long long)p.width);
    };
    long long tok = 0, fresh = 0;
    for (int r = r0; r < r1; ++r) {
        const long long old = max(p.old_lens[r], 0), add = max(p.new_lens[r], 0);
        tok += add;
        fresh += pages(old + add) - pages(old);
    }
    long long a = tok, b = fresh;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) { a += x; b += y; }
    }
    if (lane == 31) { wsum[0][warp] = a; wsum[1][warp] = b; }
    __syncthreads();
    for (int w = 0; w < warp; ++w) { a += wsum[0][w]; b += wsum[1][w]; }
    a -= tok;
    b -= fresh;
    for (int r = r0; r < r1; ++r) {
        const long long old = max(p.old_lens[r], 0), add = max(p.new_lens[r], 0);
        cu[r] = saturate(a);
        pre[r] = saturate(b);
        if (blockIdx.x == 0) {
            p.cu[r] = saturate(a);
            p.kv_lens[r] = saturate(old + add);
        }
        a += add;
        b += pages(old + add) - pages(old);
        if (r == p.R - 1) {
            cu[p.R] = saturate(a);
            pre[p.R] = saturate(b);
            if (blockIdx.x == 0) {
                p.cu[p.R] = saturate(a);
                p.pages_used[0] = saturate(b);
            }
        }
    }
    __syncthreads();
    const int at = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;
    for (int j = at; j < pre[p.R]; j += step) {
        const int r = upper_index(pre, p.R, j);   // last r with pre[r] <= j: it has fresh pages
        const int col = pages(max(p.old_lens[r], 0)) + j - pre[r];
        p.table[(size_t)r * p.table_stride + col] = j < p.num_free ? p.free_pages[j] : -1;
    }
    for (int t = at; t < p.T; t += step) {
        long long slot = -1;
        int pos = 0;
        if (t < cu[p.R]) {
            const int r = upper_index(cu, p.R, t);
            const int old = max(p.old_lens[r], 0);
            const long long at_pos = (long long)old + (t - cu[r]);
            const long long col = at_pos / p.ps;
            int page = -1;
            if (col < p.width) {
                const int have = pages(old);
                if (col < have) {
                    page = p.table[(size_t)r * p.table_stride + col];
                } else {
                    const long long j = (long long)pre[r] + col - have;
                    if (j < p.num_free) page = p.free_pages[j];
                }
            }
            pos = saturate(at_pos);
            if (page >= 0) slot = (long long)page * p.ps + at_pos % p.ps;
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
}

constexpr int kWriteThreads = 256;
constexpr int kWriteUnroll = 4;

// Blocks take whole tokens (one at least), threads 16-byte pieces of K and of V, a thread's
// loads before its first store.  Bound by memory: each row is read once and written once
// (16384 tokens of 8 heads, 134 MB: 23.4 us, 5.7 TB/s; launched after its predecessor's end
// 25.0 us, with 64-bit divisions 26.6 us besides).
// Page and row sizes are powers of two but the number of heads is not: the one division left
// is of 32-bit numbers.
__global__ void __launch_bounds__(kWriteThreads) k_paged_write(PagedWriteArgs p, int tokens) {
    const int per_head_log2 = 28 - __clz(p.d), per_tok = p.hkv << per_head_log2, ps_log2 = 31 - __clz(p.ps);
    const int t0 = blockIdx.x * tokens, n = min(tokens, p.T - t0) * per_tok;
    release_dependents();
    depend();
    for (int first = threadIdx.x; first < n; first += kWriteThreads * kWriteUnroll) {
        uint4 kv[kWriteUnroll][2];
        long long dst[kWriteUnroll];
#pragma unroll
        for (int u = 0; u < kWriteUnroll; ++u) {
            const int i = first + u * kWriteThreads;
            dst[u] = -1;
            if (i >= n) continue;
            const int tl = i / per_tok, rem = i - tl * per_tok, t = t0 + tl;
            const int h = rem >> per_head_log2, c = (rem - (h << per_head_log2)) * 8;
            const long long slot = p.slots[t];
            if (slot < 0 || slot >= ((long long)p.num_pages << ps_log2)) continue;
            const long long page = slot >> ps_log2;
            dst[u] = page * p.page_stride + (slot & (p.ps - 1)) * p.token_stride + h * p.head_stride + c;
            kv[u][0] = *reinterpret_cast<const uint4*>(p.k + t * p.k_token_stride + h * p.k_head_stride + c);
            kv[u][1] = *reinterpret_cast<const uint4*>(p.v + t * p.v_token_stride + h * p.v_head_stride + c);
        }
#pragma unroll
        for (int u = 0; u < kWriteUnroll; ++u) {
            if (dst[u] < 0) continue;
            *reinterpret_cast<uint4*>(p.k_cache + dst[u]) = kv[u][0];
            *reinterpret_cast<uint4*>(p.v_cache + dst[u]) = kv[u][1];
        }
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedPlanArgs& p, int num_sms, cudaStream_t stream) {
    const int items = std::max(p.T, 1);
    const int grid = std::min(num_sms, (items + kPlanThreads - 1) / kPlanThreads);
    const size_t smem = sizeof(int) * 2 * ((size_t)p.R + 1);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k_paged_plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(k_paged_plan, grid, kPlanThreads, smem, stream, p);
}

cudaError_t launch_paged_write(const PagedWriteArgs& p, cudaStream_t stream) {
    const long long per_tok = (long long)p.hkv * (p.d / 8);
    if (per_tok >= (1ll << 30)) return cudaErrorInvalidValue;
    const int tokens = (int)std::max(1ll, kWriteThreads * kWriteUnroll / per_tok);
    return launch_dependent(k_paged_write, (p.T + tokens - 1) / tokens, kWriteThreads, 0, stream, p, tokens);
}

}  // namespace nsa
