// paged_attn.cu -- attention of new tokens over a paged K/V cache, over all of the
// visible keys or over the key blocks that each (token, KV head) selects.
#include <math_constants.h>

#include "nsa_common.cuh"
#include "nsa_kernels.h"

namespace nsa {
namespace {

template <int F16, int D>
__global__ void __launch_bounds__(256) k_paged_rows(PagedAttnArgs p) {
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= p.T * p.hq) return;
    const int t = row / p.hq, h = row - t * p.hq, g = h / p.G;
    if (t < __ldg(p.cu) || t >= __ldg(p.cu + p.R)) return;
    const int r = seq_of_token(p.cu, p.R, t);
    const int qlen = __ldg(p.cu + r + 1) - __ldg(p.cu + r);
    if ((qlen < 0 || __ldg(p.cu + r + 1) > p.T) && lane == 0)
        record_error(p.st, NSA_ERR_BAD_INDEX, 202, r);
    const int kvlen = __ldg(p.kv_lens + r);
    if (kvlen > p.table_width * p.ps && lane == 0) record_error(p.st, NSA_ERR_BAD_INDEX, 200, r);
    const int kv = min(max(kvlen, 0), p.table_width * p.ps);
    const int pos = kv - qlen + t - __ldg(p.cu + r);
    constexpr int E = D / 32;
    float q[E], o[E];
    const uint16_t* qp = p.q + t * p.q_token_stride + h * p.q_head_stride + lane * E;
    auto cvt = [](uint16_t x) { return F16 ? __half2float(__ushort_as_half(x)) : __bfloat162float(__ushort_as_bfloat16(x)); };
    for (int e = 0; e < E; ++e) { q[e] = cvt(qp[e]); o[e] = 0.f; }
    float m = -CUDART_INF_F, l = 0.f;
    auto key = [&](int j) {
        const int page = __ldg(p.table + (size_t)r * p.table_stride + j / p.ps);
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) record_error(p.st, NSA_ERR_BAD_INDEX, 201, r, j);
            return;
        }
        const size_t at = page * p.page_stride + (j % p.ps) * p.token_stride + g * p.head_stride + lane * E;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += q[e] * cvt(p.k[at + e]);
        for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= p.scale_log2;
        const float mx = fmaxf(m, s), a = ex2_approx(m - mx), w = ex2_approx(s - mx);
        l = l * a + w;
        m = mx;
        for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * cvt(p.v[at + e]);
    };
    const int lo = p.swin > 0 ? max(0, pos - p.swin + 1) : 0, hi = min(pos, kv - 1);
    if (p.bidx) {
        for (int s = 0; s < p.topk; ++s) {
            const int b = __ldg(p.bidx + ((size_t)t * p.hkv + g) * p.topk + s);
            if (b < 0 || b > hi / p.bs) continue;
            for (int j = max(lo, b * p.bs); j <= min(hi, b * p.bs + p.bs - 1); ++j) key(j);
        }
    } else {
        for (int j = lo; j <= hi; ++j) key(j);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint16_t* op = p.out + ((size_t)t * p.hq + h) * D + lane * E;
    for (int e = 0; e < E; ++e) {
        const uint32_t u = pack2<F16>(o[e] * inv, 0.f);
        op[e] = (uint16_t)u;
    }
    if (p.lse && lane == 0)
        p.lse[(size_t)h * p.T + t] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -CUDART_INF_F;
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnArgs& p, int f16, int num_sms, cudaStream_t stream) {
    const int grid = (int)(((long long)p.T * p.hq + 7) / 8);
    if (p.d == 64) {
        if (f16) k_paged_rows<1, 64><<<grid, 256, 0, stream>>>(p);
        else k_paged_rows<0, 64><<<grid, 256, 0, stream>>>(p);
    } else {
        if (f16) k_paged_rows<1, 128><<<grid, 256, 0, stream>>>(p);
        else k_paged_rows<0, 128><<<grid, 256, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace nsa
