// paged_api.cu -- the C ABI of the paged K/V cache (include/nsa_sel.h): argument checks
// before any launch, then the launches of paged.cu and paged_attn.cu.
#include "paged.h"

using namespace nsa;

namespace {

constexpr int kMaxSeqs = 16384;   // the request lengths are scanned in shared memory

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// A stride over `size` places, of at least `least` elements; over one place it is never used.
bool stride_ok(int64_t x, int64_t size, int64_t least) { return size <= 1 || (x >= least && (x & 7) == 0); }

bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

// least_stride: 0 where rows are read (one row may stand for many), 1 where they are written.
nsa_status_t check_cache(const nsa_paged_cache_t* c, int64_t least_stride) {
    if (!c || !c->k || !c->v) return NSA_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->hkv < 1 || c->head_dim < 1 || c->page_size < 1) return NSA_ERR_INVALID_ARG;
    if (!page_size_ok(c->page_size) || (c->head_dim != 64 && c->head_dim != 128))
        return NSA_ERR_UNSUPPORTED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return NSA_ERR_INVALID_ARG;
    if (!stride_ok(c->page_stride, c->num_pages, least_stride) ||
        !stride_ok(c->token_stride, c->page_size, least_stride) || !stride_ok(c->head_stride, c->hkv, least_stride))
        return NSA_ERR_INVALID_ARG;
    return NSA_OK;
}

nsa_status_t attn_impl(const void* q, int64_t q_token_stride, int64_t q_head_stride, int T, int hq,
                       const nsa_paged_cache_t* c, const int32_t* cu, const int32_t* kv_lens, int R,
                       const int32_t* table, int width, int64_t table_stride, const int32_t* bidx,
                       int topk, int bs, float scale, int swin, void* out, float* lse, void* ws,
                       size_t ws_bytes, nsa_stream_t stream_, unsigned flags) {
    nsa_status_t s = check_cache(c, 0);
    if (s != NSA_OK) return s;
    if (flags & ~(unsigned)(NSA_F16 | NSA_TEST_SKIP_ARRIVE)) return NSA_ERR_INVALID_ARG;
    if (T < 0 || hq < 1 || R < 1 || width < 1 || table_stride < width || hq % c->hkv != 0)
        return NSA_ERR_INVALID_ARG;
    if (nsa_sel_paged_attn_workspace_size(T, R, hq, c->hkv, c->head_dim) == 0)
        return NSA_ERR_UNSUPPORTED;
    if ((long long)width * c->page_size >= (1ll << 31)) return NSA_ERR_UNSUPPORTED;
    if (!cu || !kv_lens || !table || !ws || (T > 0 && (!q || !out))) return NSA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(cu, 4) ||
        !aligned(kv_lens, 4) || !aligned(table, 4) || !aligned(bidx, 4) || !aligned(ws, 256))
        return NSA_ERR_INVALID_ARG;
    if (T > 0 && (!stride_ok(q_token_stride, T, 0) || !stride_ok(q_head_stride, hq, 0)))
        return NSA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < 1e30f) || swin < 0) return NSA_ERR_INVALID_ARG;
    if (ws_bytes < nsa_sel_paged_attn_workspace_size(T, R, hq, c->hkv, c->head_dim))
        return NSA_ERR_WORKSPACE;
    int num_sms = 0;
    if ((s = check_device(&num_sms, stream_)) != NSA_OK) return s;
    const LaunchLock lock(ws);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    DevStatus* st = static_cast<DevStatus*>(ws);
    if (T == 0)
        return cudaMemsetAsync(st, 0, sizeof(DevStatus), stream) == cudaSuccess ? NSA_OK : NSA_ERR_CUDA;
    PagedAttnArgs p{};
    p.q = static_cast<const uint16_t*>(q);
    p.q_token_stride = q_token_stride;
    p.q_head_stride = q_head_stride;
    p.k = static_cast<const uint16_t*>(c->k);
    p.v = static_cast<const uint16_t*>(c->v);
    p.page_stride = c->page_stride;
    p.token_stride = c->token_stride;
    p.head_stride = c->head_stride;
    p.num_pages = c->num_pages;
    p.ps = c->page_size;
    p.T = T;
    p.R = R;
    p.hq = hq;
    p.hkv = c->hkv;
    p.G = hq / c->hkv;
    p.d = c->head_dim;
    p.cu = cu;
    p.kv_lens = kv_lens;
    p.table = table;
    p.table_width = width;
    p.table_stride = table_stride;
    p.bidx = bidx;
    p.topk = topk;
    p.bs = bs;
    // a window that no cache outgrows is none (and leaves room for sums with it)
    p.swin = (long long)swin >= (long long)width * c->page_size ? 0 : swin;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.st = st;
    p.test_skip = (flags & NSA_TEST_SKIP_ARRIVE) != 0;
    return launch_paged_attn(p, (flags & NSA_F16) ? 1 : 0, num_sms, stream) == cudaSuccess ? NSA_OK
                                                                                           : NSA_ERR_CUDA;
}

}  // namespace

extern "C" {

nsa_status_t nsa_sel_paged_plan(const int32_t* new_lens, const int32_t* cached_lens, int num_seqs,
                                const int32_t* free_pages, int num_free, int32_t* block_table,
                                int table_width, int64_t table_stride, int page_size,
                                int total_tokens, int32_t* cu_seqlens, int32_t* kv_lens,
                                int64_t* slots, int32_t* positions, int32_t* pages_used,
                                nsa_stream_t stream) {
    if (num_seqs < 1 || num_free < 0 || table_width < 1 || table_stride < table_width ||
        page_size < 1 || total_tokens < 0)
        return NSA_ERR_INVALID_ARG;
    if (!page_size_ok(page_size) || num_seqs > kMaxSeqs || total_tokens >= (1 << 25))
        return NSA_ERR_UNSUPPORTED;
    if ((long long)table_width * page_size >= (1ll << 31)) return NSA_ERR_UNSUPPORTED;
    // (the kernel counts fresh pages in 32 bits and walks them in steps of its grid's threads)
    if ((long long)num_seqs * table_width >= (1ll << 31) - (1 << 17)) return NSA_ERR_UNSUPPORTED;
    if (!new_lens || !cached_lens || !block_table || !cu_seqlens || !kv_lens || !pages_used ||
        (num_free > 0 && !free_pages) || (total_tokens > 0 && (!slots || !positions)))
        return NSA_ERR_INVALID_ARG;
    if (!aligned(new_lens, 4) || !aligned(cached_lens, 4) || !aligned(free_pages, 4) ||
        !aligned(block_table, 4) || !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4) ||
        !aligned(slots, 8) || !aligned(positions, 4) || !aligned(pages_used, 4))
        return NSA_ERR_INVALID_ARG;
    int num_sms = 0;
    nsa_status_t s = check_device(&num_sms, stream);
    if (s != NSA_OK) return s;
    PagedPlanArgs p{};
    p.new_lens = new_lens;
    p.old_lens = cached_lens;
    p.R = num_seqs;
    p.free_pages = free_pages;
    p.num_free = num_free;
    p.table = block_table;
    p.width = table_width;
    p.table_stride = table_stride;
    p.ps = page_size;
    p.T = total_tokens;
    p.cu = cu_seqlens;
    p.kv_lens = kv_lens;
    p.slots = slots;
    p.positions = positions;
    p.pages_used = pages_used;
    return launch_paged_plan(p, num_sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? NSA_OK : NSA_ERR_CUDA;
}

nsa_status_t nsa_sel_paged_write_kv(const void* k, const void* v, int64_t k_token_stride,
                                    int64_t k_head_stride, int64_t v_token_stride,
                                    int64_t v_head_stride, const int64_t* slots, int total_tokens,
                                    const nsa_paged_cache_t* cache, nsa_stream_t stream) {
    nsa_status_t s = check_cache(cache, 1);
    if (s != NSA_OK) return s;
    if (total_tokens < 0) return NSA_ERR_INVALID_ARG;
    if (total_tokens >= (1 << 25)) return NSA_ERR_UNSUPPORTED;
    if (total_tokens > 0 && (!k || !v || !slots)) return NSA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return NSA_ERR_INVALID_ARG;
    if (total_tokens > 0 &&
        (!stride_ok(k_token_stride, total_tokens, 0) || !stride_ok(v_token_stride, total_tokens, 0) ||
         !stride_ok(k_head_stride, cache->hkv, 0) || !stride_ok(v_head_stride, cache->hkv, 0)))
        return NSA_ERR_INVALID_ARG;
    int num_sms = 0;
    if ((s = check_device(&num_sms, stream)) != NSA_OK) return s;
    if (total_tokens == 0) return NSA_OK;
    PagedWriteArgs p{};
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.k_token_stride = k_token_stride;
    p.k_head_stride = k_head_stride;
    p.v_token_stride = v_token_stride;
    p.v_head_stride = v_head_stride;
    p.slots = slots;
    p.T = total_tokens;
    p.hkv = cache->hkv;
    p.d = cache->head_dim;
    p.k_cache = static_cast<uint16_t*>(cache->k);
    p.v_cache = static_cast<uint16_t*>(cache->v);
    p.num_pages = cache->num_pages;
    p.ps = cache->page_size;
    p.page_stride = cache->page_stride;
    p.token_stride = cache->token_stride;
    p.head_stride = cache->head_stride;
    return launch_paged_write(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? NSA_OK
                                                                                        : NSA_ERR_CUDA;
}

size_t nsa_sel_paged_attn_workspace_size(int total_tokens, int num_seqs, int hq, int hkv,
                                         int head_dim) {
    if (total_tokens < 0 || num_seqs < 1 || hq < 1 || hkv < 1 || hq % hkv != 0) return 0;
    if (total_tokens >= (1 << 25) || num_seqs > kMaxSeqs || hq / hkv > kMaxGroup) return 0;
    if ((head_dim != 64 && head_dim != 128) || (long long)total_tokens * hq >= (1ll << 31)) return 0;
    return paged_attn_workspace(head_dim);
}

nsa_status_t nsa_sel_paged_attn_fwd(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                    int total_tokens, int hq, const nsa_paged_cache_t* cache,
                                    const int32_t* cu_seqlens, const int32_t* kv_lens, int num_seqs,
                                    const int32_t* block_table, int table_width,
                                    int64_t table_stride, float scale, int window_size, void* out,
                                    float* lse, void* workspace, size_t workspace_bytes,
                                    nsa_stream_t stream, unsigned flags) {
    return attn_impl(q, q_token_stride, q_head_stride, total_tokens, hq, cache, cu_seqlens, kv_lens,
                     num_seqs, block_table, table_width, table_stride, nullptr, 0, 0, scale,
                     window_size, out, lse, workspace, workspace_bytes, stream, flags);
}

nsa_status_t nsa_sel_paged_sel_fwd(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                   int total_tokens, int hq, const nsa_paged_cache_t* cache,
                                   const int32_t* cu_seqlens, const int32_t* kv_lens, int num_seqs,
                                   const int32_t* block_table, int table_width,
                                   int64_t table_stride, const int32_t* block_idx, int topk,
                                   int block_size, float scale, int window_size, void* out,
                                   float* lse, void* workspace, size_t workspace_bytes,
                                   nsa_stream_t stream, unsigned flags) {
    if (topk < 1 || block_size < 1 || (total_tokens > 0 && !block_idx)) return NSA_ERR_INVALID_ARG;
    if ((block_size != 64 && block_size != 128) || topk > kMaxTopk) return NSA_ERR_UNSUPPORTED;
    if (cache && cache->hkv > 0 && (long long)total_tokens * cache->hkv * topk >= (1ll << 31))
        return NSA_ERR_UNSUPPORTED;
    return attn_impl(q, q_token_stride, q_head_stride, total_tokens, hq, cache, cu_seqlens, kv_lens,
                     num_seqs, block_table, table_width, table_stride, block_idx, topk, block_size,
                     scale, window_size, out, lse, workspace, workspace_bytes, stream, flags);
}

}  // extern "C"
