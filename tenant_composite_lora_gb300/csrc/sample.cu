// Token sampling from logits (lora_sample): temperature, top-k, top-p and
// min-p, the token by inversion of a given uniform number.
//
// With m the row's maximum and e_i = exp((l_i - m) / tau), the kept tokens
// are a prefix of the order (logit descending, index ascending): its length
// is the least of three, so a cut -- the last kept token's logit and index --
// describes it.  Masses are 64-bit fixed point, e * 2^40 (V <= 2^20 terms of
// at most 2^40), so their sums do not depend on the order.
//
// A cluster of CTAs holds a row in registers (one read of the logits): the
// maximum, then a bound below which no kept token can lie -- the top-k's
// from the threads' own maxima, min-p's from its definition, top-p's from
// the mass above a few trial bounds -- then the few candidates above it,
// gathered and sorted by one CTA, which cuts and picks.  Rows whose
// candidates are too many for that (nearly flat ones) find the cut by
// bisection over the registers, counts and masses joined over the cluster.
// Bound by the logits' bytes and the latency of the cluster's barriers.
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

// A CTA per row, for rows too long for a cluster's registers.
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

// ---------------------------------------------------------------- a cluster per row

constexpr int SC_THREADS = 512, SC_WARPS = SC_THREADS / 32;
constexpr int SC_LIST = 2048;  // candidates that are sorted
constexpr int SC_TRIALS = 3;   // trial bounds of the top-p: e >= 2^-8, 2^-14, 2^-20
constexpr int SC_MAX_CLUSTER = 16;

__device__ __forceinline__ float key_logit(uint32_t key)
{
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ u64 fixed_mass(float e) { return __float2ull_rn(e * 1099511627776.f); }

__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename V>
__device__ __forceinline__ void st_cluster(V *local, uint32_t rank, V x)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
    if constexpr (sizeof(V) == 8)
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(x) : "memory");
    else
        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}

__device__ __forceinline__ u64 ld_cluster64(const u64 *local, uint32_t rank)
{
    uint32_t a;
    u64 x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(x) : "r"(a) : "memory");
    return x;
}

struct SampleShared {
    u64 list[SC_LIST];   // this CTA's candidates: order key (inverted), index; in rank 0 then everyone's
    u64 warp64[SC_WARPS];
    uint32_t warp32[SC_WARPS];
    // words exchanged over the cluster, two sets used in turn
    u64 x64[2][8][SC_MAX_CLUSTER];
    uint32_t count;
};

__device__ __forceinline__ u64 warp_sum64(u64 v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of N words over the cluster's threads; every thread gets them.
// `turn` counts the calls: the words' two sets are used alternately, so that
// one barrier a call is enough.
template <int N>
__device__ __forceinline__ void cluster_sums(u64 (&v)[N], SampleShared &sh, int &turn, int C, uint32_t rank)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ u64 part[2][N][SC_WARPS];
    const int set = turn++ & 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const u64 w = warp_sum64(v[i]);
        if (lane == 0)
            part[set][i][warp] = w;
    }
    __syncthreads();
    if (warp < N) {
        u64 w = lane < SC_WARPS ? part[set][warp][lane] : 0;
        w = warp_sum64(w);
        if (lane < C)
            st_cluster(&sh.x64[set][warp][rank], (uint32_t)lane, w);
    }
    if (C > 1)
        cluster_sync();
    else
        __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        u64 t = 0;
        for (int r = 0; r < C; ++r)
            t += sh.x64[set][i][r];
        v[i] = t;
    }
}

// The sum over the threads and CTAs before this one, and over all.
__device__ __forceinline__ u64 cluster_before(u64 v, u64 &all, SampleShared &sh, int &turn, int C, uint32_t rank)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int set = turn++ & 1;
    u64 inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o)
            inc += x;
    }
    __syncthreads();
    if (lane == 31)
        sh.warp64[warp] = inc;
    __syncthreads();
    u64 before = inc - v, mine = 0;
    for (int w = 0; w < SC_WARPS; ++w) {
        if (w < warp)
            before += sh.warp64[w];
        mine += sh.warp64[w];
    }
    if (threadIdx.x < C)
        st_cluster(&sh.x64[set][0][rank], (uint32_t)threadIdx.x, mine);
    if (C > 1)
        cluster_sync();
    else
        __syncthreads();
    all = 0;
    for (int r = 0; r < C; ++r) {
        if (r < (int)rank)
            before += sh.x64[set][0][r];
        all += sh.x64[set][0][r];
    }
    return before;
}

// Sorts list[0 .. n) ascending (padded to a power of two by the caller's ~0).
__device__ __forceinline__ void sort_list(u64 *list, int n2)
{
    for (int size = 2; size <= n2; size <<= 1)
        for (int step = size >> 1; step > 0; step >>= 1) {
            for (int i = threadIdx.x; i < n2 / 2; i += SC_THREADS) {
                const int lo = (i / step) * 2 * step + i % step, hi = lo + step;
                const u64 a = list[lo], b = list[hi];
                if ((a > b) == ((lo & size) == 0)) {
                    list[lo] = b;
                    list[hi] = a;
                }
            }
            __syncthreads();
        }
}

// Rank 0 of a row's cluster: sh.list holds its n candidates, padded to a
// power of two.  Sorts, cuts and picks.
__device__ __noinline__ void pick_from_list(const SampleArgs &a, SampleShared &sh, int r, int n, int k, bool has_p,
                                            float p, float mp, float u, float m, float inv, u64 z_all)
{
    constexpr int PER = SC_LIST / SC_THREADS;
    const int tid = threadIdx.x;
    auto e_of = [&](float l) { return expf((l - m) * inv); };
    // exclusive sums of a thread's PER values over the block
    auto before_of = [&](u64 v, u64 &all) {
        const int lane = tid & 31, warp = tid >> 5;
        u64 inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o)
                inc += y;
        }
        __syncthreads();
        if (lane == 31)
            sh.warp64[warp] = inc;
        __syncthreads();
        u64 b = inc - v;
        all = 0;
        for (int w = 0; w < SC_WARPS; ++w) {
            if (w < warp)
                b += sh.warp64[w];
            all += sh.warp64[w];
        }
        return b;
    };
    int n2 = 2;
    while (n2 < n)
        n2 <<= 1;
    sort_list(sh.list, n2);
    const int n1 = k > 0 ? min(n, k) : n;
    float e[PER];
    u64 w[PER], sum = 0, all;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = tid * PER + i;
        e[i] = at < n1 ? e_of(key_logit(~(uint32_t)(sh.list[at] >> 32))) : 0.f;
        w[i] = fixed_mass(e[i]);
        sum += w[i];
    }
    u64 b = before_of(sum, all);
    const u64 zk = k > 0 ? all : z_all;
    const u64 need = has_p ? max((u64)1, (u64)ceil((double)fmaxf(p, 0.f) * (double)zk)) : ~0ull;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = tid * PER + i;
        mine += at < n1 && (at == 0 || (b < need && e[i] >= mp));
        b += w[i];
    }
    // (each condition holds for a prefix of the order, so counting gives its length)
    u64 kept;
    before_of((u64)mine, kept);
    const int nk = (int)kept;
    // the kept ones by index: index, then the logit's key
    u64 t[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = tid * PER + i;
        const u64 x = at < n2 ? sh.list[at] : 0;
        t[i] = at < nk ? (x << 32) | (uint32_t)~(uint32_t)(x >> 32) : ~0ull;
    }
    __syncthreads();
    int k2 = 2;
    while (k2 < nk)
        k2 <<= 1;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (tid * PER + i < k2)
            sh.list[tid * PER + i] = t[i];
    __syncthreads();
    sort_list(sh.list, k2);
    sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = tid * PER + i;
        e[i] = at < nk ? e_of(key_logit((uint32_t)sh.list[at])) : 0.f;
        w[i] = fixed_mass(e[i]);
        sum += w[i];
    }
    u64 z;
    b = before_of(sum, z);
    u64 goal = u > 0.f ? (u64)((double)u * (double)z) : 0;
    if (goal >= z)
        goal = z - 1;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (b <= goal && goal < b + w[i]) {
            a.tokens[r] = (int)(sh.list[tid * PER + i] >> 32);
            if (a.probs)
                a.probs[r] = (float)((double)e[i] / ((double)z * 0x1p-40));
        }
        b += w[i];
    }
}

template <typename T>
struct RowType;
template <>
struct RowType<float> {
    static constexpr int E = 4;  // elements of a 16-byte vector
    static constexpr uint32_t LOWEST = 0xff800000u;
};
template <>
struct RowType<__nv_bfloat16> {
    static constexpr int E = 8;
    static constexpr uint32_t LOWEST = 0xff80ff80u;
};

// NV vectors of a row in each thread's registers.  A warp's are consecutive:
// vector v of lane i is the warp's (32 v + i)-th.
template <typename T, int NV>
struct RowRegs {
    static constexpr int E = RowType<T>::E;
    uint32_t w[NV][4];

    __device__ __forceinline__ float at(int v, int j) const
    {
        if constexpr (E == 4)
            return __uint_as_float(w[v][j]);
        else
            return (j & 1) ? bf16hi(w[v][j >> 1]) : bf16lo(w[v][j >> 1]);
    }
    __device__ __forceinline__ void set(int v, int j, float x)
    {
        if constexpr (E == 4) {
            w[v][j] = __float_as_uint(x);
        } else {  // (x is a bf16)
            const uint32_t b = __float_as_uint(x);
            w[v][j >> 1] = (j & 1) ? (w[v][j >> 1] & 0xffffu) | (b & 0xffff0000u)
                                   : (w[v][j >> 1] & 0xffff0000u) | (b >> 16);
        }
    }
};

template <typename T, int NV>
__global__ void __launch_bounds__(SC_THREADS, 2) k_sample(const SampleArgs a, const int C, const int per_warp)
{
    constexpr int E = RowType<T>::E;
    __shared__ SampleShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = C > 1 ? cluster_ctarank() : 0;
    if (C > 1)  // (waited for before the first access to another CTA's shared memory: all have begun)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const int r = blockIdx.x / C, V = a.V;
    const T *row = static_cast<const T *>(a.logits) + r * a.stride;
    // vectors are taken at 16-byte boundaries: `head` elements of the first lie before the row
    const int head = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    // every warp of the cluster has per_warp vectors, so that the CTAs' shares are alike
    const int base = ((int)rank * SC_WARPS + warp) * per_warp * E - head;  // index of the warp's first element
    auto index = [&](int v, int j) { return base + (v * 32 + lane) * E + j; };
    int turn = 0;

    RowRegs<T, NV> x;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = index(v, 0);
        if (i >= 0 && i + E <= V && v * 32 + lane < per_warp) {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(row + i));
            x.w[v][0] = q.x;
            x.w[v][1] = q.y;
            x.w[v][2] = q.z;
            x.w[v][3] = q.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x.w[v][j] = RowType<T>::LOWEST;
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (i + j >= 0 && i + j < V && v * 32 + lane < per_warp)
                    x.set(v, j, (float)row[i + j]);
        }
    }
    // NaN counts as -inf, -0 as 0
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float l = x.at(v, j) + 0.f;
            l = l == l ? l : -INFINITY;
            x.set(v, j, l);
            m = fmaxf(m, l);
        }
    const float my_max = m;
    m = __uint_as_float(0u);
    {
        uint32_t k = order_key(my_max);
        k = __reduce_max_sync(0xffffffffu, k);
        if (lane == 0)
            sh.warp32[warp] = k;
        __syncthreads();
        if (C > 1)
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (warp == 0) {
            k = __reduce_max_sync(0xffffffffu, lane < SC_WARPS ? sh.warp32[lane] : 0u);
            if (lane < C)
                st_cluster(&sh.x64[1][7][rank], (uint32_t)lane, (u64)k);
        }
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
        k = 0;
        for (int q = 0; q < C; ++q)
            k = max(k, (uint32_t)sh.x64[1][7][q]);
        m = key_logit(k);
    }
    if (m == -INFINITY) {
        if (rank == 0 && tid == 0) {
            a.tokens[r] = -1;
            if (a.probs)
                a.probs[r] = 0.f;
        }
        return;  // (the whole cluster; its last DSMEM access was before the barrier)
    }
    const float tau = a.tau ? a.tau[r] : 1.f;
    if (!(tau > 0.f)) {  // the largest, of the lowest index
        uint32_t best = 0xffffffffu;
#pragma unroll
        for (int v = NV - 1; v >= 0; --v)
#pragma unroll
            for (int j = E - 1; j >= 0; --j)
                if (x.at(v, j) == m)
                    best = (uint32_t)index(v, j);
        best = __reduce_min_sync(0xffffffffu, best);
        if (lane == 0)
            sh.warp32[warp] = best;
        __syncthreads();
        if (warp == 0) {
            best = __reduce_min_sync(0xffffffffu, lane < SC_WARPS ? sh.warp32[lane] : 0xffffffffu);
            if (lane == 0)
                st_cluster(&sh.x64[0][7][rank], 0u, (u64)best);
        }
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
        if (rank == 0 && tid == 0) {
            for (int q = 0; q < C; ++q)
                best = min(best, (uint32_t)sh.x64[0][7][q]);
            a.tokens[r] = (int)best;
            if (a.probs)
                a.probs[r] = 1.f;
        }
        return;
    }
    // (a temperature beyond 1e37 or below 1e-37 counts as that: no product below is inf * 0)
    const float inv = fminf(fmaxf(1.f / tau, 1e-37f), 1e37f), c2 = inv * 1.44269504088896341f;
    float tmax = my_max;
    if (m == INFINITY) {  // the tokens at +inf share the mass
        tmax = my_max == INFINITY ? 0.f : -INFINITY;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < E; ++j)
                x.set(v, j, x.at(v, j) == INFINITY ? 0.f : -INFINITY);
        m = 0.f;
    }
    const int k = a.top_k ? a.top_k[r] : 0;
    const float p = a.top_p ? a.top_p[r] : 1.f;
    const float mp = !a.min_p || !(a.min_p[r] > 0.f) ? 0.f : fminf(a.min_p[r], 1.f);
    const float u = a.u[r];
    const bool has_k = k > 0 && k < V, has_p = p < 1.f;
    auto e_of = [&](float l) { return expf((l - m) * inv); };           // of a single token
    auto e_fast = [&](float l) { return fast_exp2((l - m) * c2); };     // in sums over many
    // below this no token has e >= min_p (with room for the roundings)
    const float l_mp = mp > 0.f ? m + (logf(mp) - 1e-3f) * (1.f / inv) : -INFINITY;

    // ---- the bound and, where it is needed, the mass of all
    float bound = -INFINITY;
    u64 z_all = 0;
    bool listed = false;  // the candidates fit the list
    if (has_k) {
        // at least k / C (rounded up) of this CTA's tokens are at or above the threads' maximum of that rank,
        // so at least k of all at or above the least of the CTAs' ones
        const int want = (k + C - 1) / C;
        uint32_t key = 0;
        const uint32_t mine = order_key(tmax);
        if (want <= SC_THREADS) {
            for (int bit = 31; bit >= 12; --bit) {  // (the lower bits make little difference)
                const uint32_t t = key | (1u << bit);
                if (__syncthreads_count(mine >= t) >= want)
                    key = t;
            }
        }
        const int set = turn++ & 1;
        if (tid < C)
            st_cluster(&sh.x64[set][0][rank], (uint32_t)tid, (u64)key);
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
        for (int q = 0; q < C; ++q)
            key = min(key, (uint32_t)sh.x64[set][0][q]);
        bound = key == 0 ? -INFINITY : key_logit(key);
        if (!(bound == bound))
            bound = -INFINITY;
        if (!has_p)
            bound = fmaxf(bound, l_mp);
        listed = true;
    } else if (has_p) {
        const float b0 = m - 8.f / c2, b1 = m - 14.f / c2, b2 = m - 20.f / c2;
        u64 s[1 + 2 * SC_TRIALS] = {};
        uint32_t n0 = 0, n1 = 0, n2 = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float t = 0.f, t0 = 0.f, t1 = 0.f, t2 = 0.f;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float l = x.at(v, j), e = e_fast(l);
                t += e;
                if (l >= b0) {
                    t0 += e;
                    ++n0;
                }
                if (l >= b1) {
                    t1 += e;
                    ++n1;
                }
                if (l >= b2) {
                    t2 += e;
                    ++n2;
                }
            }
            s[0] += fixed_mass(t);
            s[1] += fixed_mass(t0);
            s[2] += fixed_mass(t1);
            s[3] += fixed_mass(t2);
        }
        s[4] = n0;
        s[5] = n1;
        s[6] = n2;
        cluster_sums(s, sh, turn, C, rank);
        z_all = s[0];
        // (the trial masses are good to 1e-6; a bound that only just suffices is passed over)
        const double need = (double)fmaxf(p, 0.f) * (double)z_all * (1.0 + 1e-5);
        const float b[SC_TRIALS] = {b0, b1, b2};
        for (int i = 0; i < SC_TRIALS && !listed; ++i)
            if ((double)s[1 + i] >= need && s[4 + i] <= SC_LIST) {
                bound = b[i];
                listed = true;
            }
        if (!listed && mp > 0.f)
            listed = true;  // as far as min_p goes, whatever its count
        bound = fmaxf(bound, l_mp);
    }

    // ---- the candidates at or above the bound, sorted and cut by rank 0
    if (listed) {
        const int set = turn++ & 1;
        if (tid == 0)
            sh.count = 0;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float l = x.at(v, j);
                if (l >= bound && l > -INFINITY) {
                    const uint32_t at = atomicAdd(&sh.count, 1u);
                    if (at < SC_LIST)
                        sh.list[at] = ((u64)~order_key(l) << 32) | (uint32_t)index(v, j);
                }
            }
        __syncthreads();
        if (tid < C)
            st_cluster(&sh.x64[set][0][rank], (uint32_t)tid, (u64)sh.count);
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
        u64 n_all = 0;
        for (int q = 0; q < C; ++q)
            n_all += sh.x64[set][0][q];
        if (n_all <= SC_LIST) {
            if (rank == 0) {
                int n = (int)sh.x64[set][0][0];
                for (int q = 1; q < C; ++q) {
                    const int nq = (int)sh.x64[set][0][q];
                    for (int i = tid; i < nq; i += SC_THREADS)
                        sh.list[n + i] = ld_cluster64(&sh.list[i], (uint32_t)q);
                    n += nq;
                }
                int n2 = 2;
                while (n2 < n)
                    n2 <<= 1;
                for (int i = n + tid; i < n2; i += SC_THREADS)
                    sh.list[i] = ~0ull;
            }
            if (C > 1)
                cluster_sync();  // read: the other CTAs' shared memory may go
            if (rank != 0)
                return;
            __syncthreads();
            pick_from_list(a, sh, r, (int)n_all, has_k ? k : 0, has_p, p, mp, u, m, inv, z_all);
            return;
        }
    }

    // ---- too many candidates, or no bound at all: the cut by bisection over the registers
    uint32_t cut = 0;    // order key of the last kept logit
    u64 ties = ~0ull;    // how many of the tokens that equal it are kept, by index
    u64 above = 0;       // mass of the tokens above it
    auto key_at = [&](int v, int j) { return order_key(x.at(v, j)); };
    if (has_k) {
        uint32_t lo = 0;  // the largest key with at least k tokens at or above
        for (int bit = 31; bit >= (E == 8 ? 16 : 0); --bit) {
            const uint32_t t = lo | (1u << bit);
            uint32_t n = 0;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < E; ++j)
                    n += key_at(v, j) >= t;
            u64 s[1] = {n};
            cluster_sums(s, sh, turn, C, rank);
            if (s[0] >= (u64)k)
                lo = t;
        }
        cut = lo;
        if (E == 8 && !(lo >> 31))
            cut |= 0xffffu;  // a negative bf16's key ends in ones
    }
    if (has_k) {
        // mass above the cut, tokens above and at it
        u64 s[3] = {};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const uint32_t key = key_at(v, j);
                if (key > cut) {
                    t += e_fast(x.at(v, j));
                    ++s[1];
                }
                s[2] += key == cut;
            }
            s[0] += fixed_mass(t);
        }
        cluster_sums(s, sh, turn, C, rank);
        above = s[0];
        ties = min(s[2], (u64)k - s[1]);
    }
    const u64 w_cut = cut ? fixed_mass(e_of(key_logit(cut))) : 0;
    if (has_p) {
        const u64 zk = has_k ? above + ties * w_cut : z_all;
        const u64 need = max((u64)1, (u64)ceil((double)fmaxf(p, 0.f) * (double)zk));
        if (above >= need || !has_k) {  // the cut moves up: the largest key with at least `need` at or above
            uint32_t lo = 0;
            u64 over = 0;  // mass above it
            for (int bit = 31; bit >= (E == 8 ? 16 : 0); --bit) {
                const uint32_t t = lo | (1u << bit);
                u64 s[1] = {};
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float f = 0.f;
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        f += key_at(v, j) >= t && key_at(v, j) > cut ? e_fast(x.at(v, j)) : 0.f;
                    s[0] += fixed_mass(f);
                }
                cluster_sums(s, sh, turn, C, rank);
                if (s[0] >= need)
                    lo = t;
                else
                    over = s[0];
            }
            if (E == 8 && !(lo >> 31))
                lo |= 0xffffu;
            cut = max(lo, cut);
            const u64 w = fixed_mass(e_of(key_logit(cut)));
            ties = w > 0 && need > over ? (need - over + w - 1) / w : 1;
        } else if (w_cut > 0) {
            ties = min(ties, (need - above + w_cut - 1) / w_cut);
        }
    }
    // the kept masses in index order: a vector's in turn, a lane's vectors of a warp 32 apart
    int last_tie = V;
    if (ties != ~0ull) {
        // the index of the last tie kept
        u64 n = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < E; ++j)
                n += key_at(v, j) == cut;
        // (within a warp the order is vector by vector, so the warp's first lane counts for all of it)
        const u64 in_warp = warp_sum64(n);
        u64 all;
        const u64 before = __shfl_sync(0xffffffffu, cluster_before(lane == 0 ? in_warp : 0, all, sh, turn, C, rank), 0);
        uint32_t found = 0xffffffffu;
        if (all > ties && before < ties && ties <= before + in_warp) {
            u64 run = before;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                int mine = 0;
#pragma unroll
                for (int j = 0; j < E; ++j)
                    mine += key_at(v, j) == cut;
                int inc = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o)
                        inc += y;
                }
                u64 at = run + inc - mine;
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (key_at(v, j) == cut && ++at == ties)
                        found = (uint32_t)index(v, j);
                run += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        u64 s[1] = {found == 0xffffffffu ? 0ull : (u64)found + 1};
        cluster_sums(s, sh, turn, C, rank);
        if (s[0] > 0)
            last_tie = (int)s[0] - 1;
    }
    auto kept = [&](int v, int j) -> float {
        const float l = x.at(v, j);
        const uint32_t key = order_key(l);
        if (key < cut || (key == cut && index(v, j) > last_tie))
            return 0.f;
        const float e = e_fast(l);
        return l == m || e >= mp ? e : 0.f;
    };
    auto vector_mass = [&](int v) {
        float f = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j)
            f += kept(v, j);
        return fixed_mass(f);
    };
    u64 in_lane = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
        in_lane += vector_mass(v);
    const u64 in_warp = warp_sum64(in_lane);
    u64 z;
    const u64 before = __shfl_sync(0xffffffffu, cluster_before(lane == 0 ? in_warp : 0, z, sh, turn, C, rank), 0);
    u64 goal = u > 0.f ? (u64)((double)u * (double)z) : 0;
    if (goal >= z)
        goal = z - 1;
    if (before <= goal && goal < before + in_warp) {
        u64 run = before;
        bool done = false;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const u64 mine = vector_mass(v);
            u64 inc = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o)
                    inc += y;
            }
            const u64 at = run + inc - mine;
            if (!done && at <= goal && goal < run + inc) {
                // this lane's vector: its elements in turn; the last kept one if their sum falls short
                float f = 0.f;
                const float want = (float)((double)(goal - at) * 0x1p-40);
                int pick = -1;
                float pe = 0.f;
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float e = kept(v, j);
                    if (e > 0.f && (pick < 0 || f <= want)) {
                        pick = index(v, j);
                        pe = e_of(x.at(v, j));
                    }
                    f += e;
                }
                a.tokens[r] = pick;
                if (a.probs)
                    a.probs[r] = (float)((double)pe / ((double)z * 0x1p-40));
                done = true;
            }
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
}

template <typename T, int NV>
cudaError_t launch_cluster(const SampleArgs &a, int T_rows, int C, int per_warp, cudaStream_t st)
{
    if (C > 8) {
        static thread_local int attr_dev = -1;  // per host thread
        int dev = 0;
        cudaGetDevice(&dev);
        if (attr_dev != dev) {
            const cudaError_t e = cudaFuncSetAttribute(k_sample<T, NV>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess)
                return e;
            attr_dev = dev;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)T_rows * C, 1, 1);
    cfg.blockDim = dim3(SC_THREADS, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_sample<T, NV>, a, C, per_warp);
}

// The cluster's size and the vectors a thread holds: as few CTAs as hold a
// row in 16 or 32 registers a thread; while the rows leave SMs idle, twice as
// many.  Rows too long for 16 CTAs take the CTA-per-row kernel.
template <typename T>
cudaError_t launch_sample(const SampleArgs &a, int T_rows, cudaStream_t st)
{
    constexpr int E = RowType<T>::E, MOST = E == 8 ? 4 : 8;
    const int vectors = (a.V + E - 1) / E + 1;  // (a row may begin inside one)
    int C = 1;
    while (C < SC_MAX_CLUSTER && vectors > C * SC_THREADS * MOST)
        C *= 2;
    if (vectors > C * SC_THREADS * MOST || (long long)T_rows * C > 0x7fffffffll) {
        k_sample_simple<T><<<T_rows, SA_THREADS, 0, st>>>(a);
        return cudaGetLastError();
    }
    while (C < SC_MAX_CLUSTER && vectors > C * SC_THREADS && (long long)T_rows * C * 2 <= sm_count())
        C *= 2;
    const int per_warp = (vectors + C * SC_WARPS - 1) / (C * SC_WARPS), per = (per_warp + 31) / 32;
    if (per <= 1)
        return launch_cluster<T, 1>(a, T_rows, C, per_warp, st);
    if (per <= 2)
        return launch_cluster<T, 2>(a, T_rows, C, per_warp, st);
    if (per <= 4)
        return launch_cluster<T, 4>(a, T_rows, C, per_warp, st);
    if constexpr (MOST == 8)
        return launch_cluster<T, 8>(a, T_rows, C, per_warp, st);
    return cudaErrorInvalidValue;  // (not reached: per <= MOST)
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
    const cudaError_t e = logits_type == LORA_TYPE_F32 ? launch_sample<float>(a, T, st)
                                                       : launch_sample<__nv_bfloat16>(a, T, st);
    return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
