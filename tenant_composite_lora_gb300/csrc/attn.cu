// Attention over the paged cache for a planned batch (lora_prefix_attention).
//
//     out = sum_j softmax_j(scale q . k_j) v_j     over the group's prefix, then the request's own
//                                                  tokens up to the query itself
#include "attn.h"
#include "ptx.cuh"

namespace tcl {

namespace {

// A warp per (query token, head): lanes share the head's elements, the
// softmax runs over the keys in order.
template <int D>
__global__ void __launch_bounds__(256) k_attn_simple(const AttnPlanDev p, const AttnArgs a)
{
    constexpr int E = D / 32;
    const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (w >= (long long)a.TQ * p.hq)
        return;
    const int t = (int)(w / p.hq), h = (int)(w % p.hq), hk = h / (p.hq / p.hkv);
    const int b = p.tok_req[t];
    float q[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(a.q[t * a.q_stride + (long long)h * D + lane * E + e]) * a.scale;
        acc[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    if (b >= 0) {
        const int n = p.q_off[b + 1] - p.q_off[b], i = t - p.q_off[b];
        const int g = p.grp[b];
        const int lens[2] = {g >= 0 ? p.p_len[g] : 0, max(0, min(p.s_len[b], p.s_len[b] - n + i + 1))};
        const int32_t *tab[2] = {p.p_pages + (long long)max(g, 0) * p.max_ppages,
                                 p.s_pages + (long long)b * p.max_spages};
        for (int part = 0; part < 2; ++part)
            for (int j = 0; j < lens[part]; ++j) {
                const int pg = tab[part][j >> p.page_log2];
                if (pg < 0)
                    continue;
                const long long off =
                    (((long long)pg * p.hkv + hk) * p.page + (j & (p.page - 1))) * D + lane * E;
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    s = fmaf(q[e], __bfloat162float(a.k[off + e]), s);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    s += __shfl_xor_sync(0xffffffffu, s, o);
                const float mn = fmaxf(m, s);
                if (mn == -INFINITY)
                    continue;
                const float c = expf(m - mn), w0 = expf(s - mn);
                l = l * c + w0;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[e] = acc[e] * c + w0 * __bfloat162float(a.v[off + e]);
                m = mn;
            }
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
#pragma unroll
    for (int e = 0; e < E; ++e)
        a.out[t * a.out_stride + (long long)h * D + lane * E + e] = __float2bfloat16_rn(acc[e] * inv);
    if (a.lse && lane == 0)
        a.lse[w] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_attn(const AttnPlanDev &p, const AttnArgs &a, cudaStream_t st)
{
    const long long warps = (long long)a.TQ * p.hq;
    const unsigned grid = (unsigned)((warps + 7) / 8);
    if (p.d == 64)
        k_attn_simple<64><<<grid, 256, 0, st>>>(p, a);
    else
        k_attn_simple<128><<<grid, 256, 0, st>>>(p, a);
    return cudaGetLastError();
}

}  // namespace tcl

using namespace tcl;

extern "C" {

lora_status lora_prefix_attention(const void *q_dev, long long q_stride, void *out_dev, long long out_stride,
                                  float *lse_dev, const lora_kv_cache *cache, lora_attn_plan *plan, float scale,
                                  lora_stream_t stream)
{
    if (!cache || !plan || !plan->built)
        return LORA_ERR_INVALID_ARG;
    const AttnPlanDev &p = plan->dev;
    if (cache->page_size != p.page || cache->hkv != p.hkv || cache->d != p.d || cache->num_pages < plan->num_pages)
        return LORA_ERR_INVALID_ARG;
    if (plan->TQ == 0)
        return LORA_OK;  // (arrays of no elements may have no address)
    const long long row = (long long)p.hq * p.d;
    if (!q_dev || !out_dev || q_dev == out_dev || q_stride < row || out_stride < row || q_stride % 8 || out_stride % 8 ||
        ((reinterpret_cast<uintptr_t>(q_dev) | reinterpret_cast<uintptr_t>(out_dev)) & 15u))
        return LORA_ERR_INVALID_ARG;
    AttnArgs a{};
    a.q = static_cast<const __nv_bfloat16 *>(q_dev);
    a.out = static_cast<__nv_bfloat16 *>(out_dev);
    a.lse = lse_dev;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.k = cache->k;
    a.v = cache->v;
    a.scale = scale;
    a.TQ = plan->TQ;
    return launch_attn(p, a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
