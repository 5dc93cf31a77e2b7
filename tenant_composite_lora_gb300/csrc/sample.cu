// Token sampling from logits (lora_sample): temperature, top-k, top-p and
// min-p, the token by inversion of a given uniform number.
//
// With m the row's maximum and e_i = exp((l_i - m) / tau), the kept tokens
// are a prefix of the order (logit descending, index ascending): its length
// is the least of three, so a cut -- a logit, and how many of the tokens
// that equal it -- describes it.  Masses are 64-bit fixed point, e * 2^40:
// their sums are exact (V <= 2^20 terms of at most 2^40), so they are the
// same whatever the order, and the cut and the token follow from them alone.
#include "internal.h"
#include "ptx.cuh"

namespace tcl {

namespace {

constexpr int SA_THREADS = 1024;

struct SampleArgs {
    const void *logits;
    const float *u, *tau, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens;
    float *probs;
    long long stride;
    int V;
};

typedef unsigned long long u64;

template <typename T>
__device__ __forceinline__ float load_logit(const T *row, int i);
template <>
__device__ __forceinline__ float load_logit<float>(const float *row, int i)
{
    const float l = row[i] + 0.f;  // -0 counts as 0
    return isnan(l) ? -INFINITY : l;
}
template <>
__device__ __forceinline__ float load_logit<__nv_bfloat16>(const __nv_bfloat16 *row, int i)
{
    const float l = __bfloat162float(row[i]) + 0.f;
    return isnan(l) ? -INFINITY : l;
}

// Unsigned integers in the order of the floats.
__device__ __forceinline__ uint32_t order_key(float l)
{
    const uint32_t b = __float_as_uint(l);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

struct RowScale {
    float m, inv;
    __device__ __forceinline__ float e(float l) const
    {
        return l == -INFINITY ? 0.f : l == m ? 1.f : expf((l - m) * inv);
    }
    __device__ __forceinline__ u64 mass(float l) const { return __float2ull_rn(e(l) * 1099511627776.f); }
};

template <typename V>
__device__ V block_sum(V v, V *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        sh[threadIdx.x >> 5] = v;
    __syncthreads();
    V r = 0;
    for (int w = 0; w < SA_THREADS / 32; ++w)
        r += sh[w];
    return r;
}

// Exclusive sum over the threads before this one.
template <typename V>
__device__ V block_before(V v, V *sh)
{
    const int lane = threadIdx.x & 31;
    V inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o)
            inc += x;
    }
    __syncthreads();
    if (lane == 31)
        sh[threadIdx.x >> 5] = inc;
    __syncthreads();
    V r = inc - v;
    for (int w = 0; w < (int)(threadIdx.x >> 5); ++w)
        r += sh[w];
    return r;
}

// A CTA per row.
template <typename T>
__global__ void __launch_bounds__(SA_THREADS) k_sample_simple(const SampleArgs a)
{
    __shared__ u64 sh[32], hist[256];
    __shared__ float shf[32];
    __shared__ u64 s_run;
    __shared__ uint32_t s_key;
    __shared__ int s_idx;
    const int r = blockIdx.x, tid = threadIdx.x, V = a.V;
    const T *row = static_cast<const T *>(a.logits) + r * a.stride;

    float m = -INFINITY;
    for (int i = tid; i < V; i += SA_THREADS)
        m = fmaxf(m, load_logit(row, i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0)
        shf[tid >> 5] = m;
    __syncthreads();
    for (int w = 0; w < SA_THREADS / 32; ++w)
        m = fmaxf(m, shf[w]);
    if (m == -INFINITY) {
        if (tid == 0) {
            a.tokens[r] = -1;
            if (a.probs)
                a.probs[r] = 0.f;
        }
        return;
    }
    const float tau = a.tau ? a.tau[r] : 1.f;
    const bool greedy = !(tau > 0.f);
    const RowScale sc{m, greedy ? 1.f : 1.f / tau};
    const int k = greedy ? 1 : a.top_k ? a.top_k[r] : 0;
    const float p = greedy || !a.top_p ? 1.f : a.top_p[r];
    const float mp = greedy || !a.min_p || !(a.min_p[r] > 0.f) ? 0.f : fminf(a.min_p[r], 1.f);

    // first k: the cut's key and how many of its ties stay
    uint32_t cut = 0;
    u64 ties = ~0ull;  // all
    if (k > 0 && k < V) {
        u64 need = (u64)k;
        uint32_t pre = 0;
        for (int sft = 24; sft >= 0; sft -= 8) {
            if (tid < 256)
                hist[tid] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += SA_THREADS) {
                const uint32_t key = order_key(load_logit(row, i));
                if (sft == 24 || (key >> (sft + 8)) == (pre >> (sft + 8)))
                    atomicAdd(&hist[(key >> sft) & 255], 1ull);
            }
            __syncthreads();
            if (tid == 0) {
                int b = 255;
                while (hist[b] < need)
                    need -= hist[b--];
                s_key = pre | ((uint32_t)b << sft);
                s_run = need;
            }
            __syncthreads();
            pre = s_key;
            need = s_run;
        }
        cut = pre;
        ties = need;
    }
    // mass of those, then the shortest prefix of them that reaches top_p of it
    u64 above = 0, equal = 0;
    float cut_l = -INFINITY;
    if (cut) {
        const uint32_t b = cut ^ ((cut >> 31) ? 0x80000000u : 0xffffffffu);
        cut_l = __uint_as_float(b);
    }
    for (int i = tid; i < V; i += SA_THREADS) {
        const float l = load_logit(row, i);
        const uint32_t key = order_key(l);
        if (key > cut)
            above += sc.mass(l);
        equal += key == cut;
    }
    above = block_sum(above, sh);
    equal = block_sum(equal, sh);
    if (ties > equal)
        ties = equal;
    const u64 zk = above + ties * sc.mass(cut_l);
    if (p < 1.f) {
        u64 need = p > 0.f ? (u64)ceil((double)p * (double)zk) : 1ull;
        if (need < 1)
            need = 1;
        if (above >= need) {  // the cut moves up
            uint32_t pre = 0;
            const uint32_t kcut = cut;
            for (int sft = 24; sft >= 0; sft -= 8) {
                if (tid < 256)
                    hist[tid] = 0;
                __syncthreads();
                for (int i = tid; i < V; i += SA_THREADS) {
                    const float l = load_logit(row, i);
                    const uint32_t key = order_key(l);
                    if (key > kcut && (sft == 24 || (key >> (sft + 8)) == (pre >> (sft + 8))))
                        atomicAdd(&hist[(key >> sft) & 255], sc.mass(l));
                }
                __syncthreads();
                if (tid == 0) {
                    int b = 255;
                    while (hist[b] < need)
                        need -= hist[b--];
                    s_key = pre | ((uint32_t)b << sft);
                    s_run = need;
                }
                __syncthreads();
                pre = s_key;
                need = s_run;
            }
            cut = pre;
            const u64 w = sc.mass(__uint_as_float(cut ^ ((cut >> 31) ? 0x80000000u : 0xffffffffu)));
            ties = (need + w - 1) / w;
        } else {
            const u64 w = sc.mass(cut_l);
            if (w > 0) {
                const u64 t = (need - above + w - 1) / w;
                ties = t < ties ? t : ties;
            }
        }
    }
    // ties stay by index: the last one's index; then the masses in index order
    const int per = (V + SA_THREADS - 1) / SA_THREADS, i0 = min(V, tid * per), i1 = min(V, i0 + per);
    u64 mine = 0;
    for (int i = i0; i < i1; ++i)
        mine += order_key(load_logit(row, i)) == cut;
    const u64 before = block_before(mine, sh);
    if (tid == 0)
        s_idx = ties == 0 ? -1 : V;
    __syncthreads();
    if (ties > 0 && before < ties && ties <= before + mine) {
        u64 n = before;
        for (int i = i0; i < i1; ++i)
            if (order_key(load_logit(row, i)) == cut && ++n == ties) {
                s_idx = i;
                break;
            }
    }
    __syncthreads();
    const int last_tie = s_idx;
    auto kept_mass = [&](int i) -> u64 {
        const float l = load_logit(row, i);
        const uint32_t key = order_key(l);
        if (key < cut || (key == cut && i > last_tie))
            return 0;
        const float e = sc.e(l);
        return e >= mp ? __float2ull_rn(e * 1099511627776.f) : 0;
    };
    u64 seg = 0;
    for (int i = i0; i < i1; ++i)
        seg += kept_mass(i);
    const u64 z = block_sum(seg, sh);
    const u64 run0 = block_before(seg, sh);
    const float u = a.u[r];
    u64 goal = u > 0.f ? (u64)((double)u * (double)z) : 0;
    if (goal >= z)
        goal = z - 1;
    if (run0 <= goal && goal < run0 + seg) {
        u64 c = run0;
        for (int i = i0; i < i1; ++i) {
            c += kept_mass(i);
            if (c > goal) {
                a.tokens[r] = i;
                if (a.probs)
                    a.probs[r] = (float)((double)sc.e(load_logit(row, i)) / ((double)z * 0x1p-40));
                break;
            }
        }
    }
}

}  // namespace

}  // namespace tcl

using namespace tcl;

extern "C" {

lora_status lora_sample(const void *logits_dev, int logits_type, long long row_stride, int T, int V,
                        const float *u_dev, const float *temperature_dev, const int32_t *top_k_dev,
                        const float *top_p_dev, const float *min_p_dev, int32_t *tokens_dev, float *probs_dev,
                        lora_stream_t stream)
{
    if (T < 0 || V < 1 || row_stride < V ||
        (logits_type != LORA_TYPE_F32 && logits_type != LORA_TYPE_BF16))
        return LORA_ERR_INVALID_ARG;
    if (V > LORA_MAX_VOCAB || T > LORA_MAX_TOKENS)
        return LORA_ERR_NOT_SUPPORTED;
    if (T == 0)
        return LORA_OK;  // (arrays of no elements may have no address)
    if (!logits_dev || !u_dev || !tokens_dev ||
        (reinterpret_cast<uintptr_t>(logits_dev) & (logits_type == LORA_TYPE_F32 ? 3u : 1u)))
        return LORA_ERR_INVALID_ARG;
    const SampleArgs a{logits_dev, u_dev, temperature_dev, top_p_dev, min_p_dev, top_k_dev, tokens_dev, probs_dev,
                       row_stride, V};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (logits_type == LORA_TYPE_F32)
        k_sample_simple<float><<<T, SA_THREADS, 0, st>>>(a);
    else
        k_sample_simple<__nv_bfloat16><<<T, SA_THREADS, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
