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
// gathered by one CTA, which cuts and picks.  Rows whose
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

// x in [0, 1) as a 64-bit fraction (exact from 2^-40 on), in two exact parts.
// (No arithmetic here is in double: an SM does two such products a clock.)
__device__ __forceinline__ u64 fraction(float x)
{
    const float y = x * 4294967296.f;
    const uint32_t hi = __float2uint_rz(y);
    return ((u64)hi << 32) | __float2uint_rz((y - __uint2float_rz(hi)) * 4294967296.f);
}

// The mass that a prefix has to reach for top_p of zk: p zk rounded up, at least 1.
__device__ __forceinline__ u64 needed_mass(float p, u64 zk)
{
    if (!(p > 0.f))
        return 1;
    const u64 f = fraction(p), n = __umul64hi(f, zk) + (f * zk != 0);
    return n ? n : 1;
}

// The token is the one whose cumulative mass first exceeds this: u z rounded down.
__device__ __forceinline__ u64 goal_mass(float u, u64 z)
{
    if (!(u > 0.f))
        return 0;
    return u < 1.f ? __umul64hi(fraction(u), z) : z - 1;
}

__device__ __forceinline__ float share(float e, u64 z) { return e / (__ull2float_rn(z) * 0x1p-40f); }

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
        const u64 need_of_zk = needed_mass(p, zk);
        u64 need = need_of_zk;
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
    const u64 goal = goal_mass(u, z);
    if (run0 <= goal && goal < run0 + seg) {
        u64 c = run0;
        for (int i = i0; i < i1; ++i) {
            c += kept_mass(i);
            if (c > goal) {
                a.tokens[r] = i;
                if (a.probs)
                    a.probs[r] = share(sc.e(load_logit(row, i)), z);
                break;
            }
        }
    }
}

// ---------------------------------------------------------------- a cluster per row

constexpr int SC_THREADS = 512, SC_WARPS = SC_THREADS / 32;
constexpr int SC_LIST = 2048;   // candidates that one CTA takes
constexpr int SC_SLOTS = 4096;  // places for them, an equal share for each CTA of the cluster
constexpr int SC_TRIALS = 3;   // trial bounds of the top-p: e >= 2^-8, 2^-14, 2^-20
constexpr int SC_MAX_CLUSTER = 16;
static_assert(SC_MAX_CLUSTER <= SC_WARPS, "a warp moves a CTA's candidates");

__device__ __forceinline__ float key_logit(uint32_t key)
{
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// e * 2^40 rounded down, for 0 <= e < 2^15: in two exact parts of 32 bits.
__device__ __forceinline__ u64 fixed_mass(float e)
{
    const float x = e * 65536.f;
    const uint32_t hi = __float2uint_rz(x);
    const uint32_t lo = __float2uint_rz((x - __uint2float_rz(hi)) * 16777216.f);
    return ((u64)hi << 24) + lo;
}

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

struct SampleShared {
    // rank 0: the candidates (order key inverted, index), SC_SLOTS / C places for each CTA's; then all in a row
    alignas(16) u64 slots[SC_SLOTS];
    alignas(16) u64 list[SC_LIST];
    alignas(16) u64 mass[SC_THREADS];  // theirs, where they are few
    u64 warp64[SC_WARPS];
    uint32_t warp32[SC_WARPS];
    uint32_t packed[2][SC_WARPS];
    // words exchanged over the cluster, two sets used in turn
    u64 x64[2][8][SC_MAX_CLUSTER];
    u64 part[2][8][SC_WARPS];
    uint32_t count;
};
// (dynamic shared memory, whose address space functions that are not inlined know too)
__device__ __forceinline__ SampleShared &sample_shared()
{
    extern __shared__ __align__(16) unsigned char sample_smem[];
    return *reinterpret_cast<SampleShared *>(sample_smem);
}

__device__ __forceinline__ u64 warp_sum64(u64 v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of N words over the cluster's threads (WARP: its warps, whose lanes
// hold the same); every thread gets them.
// `turn` counts the calls: the words' two sets are used alternately, so that
// one barrier a call is enough.
template <bool WARP, int N>
__device__ __forceinline__ void cluster_sums(u64 (&v)[N], SampleShared &sh, int &turn, int C, uint32_t rank)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int set = turn++ & 1;
    auto &part = sh.part;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const u64 w = WARP ? v[i] : warp_sum64(v[i]);
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

// Sum over the block of a value, to all threads.
__device__ __forceinline__ u64 block_sum64(u64 v, SampleShared &sh)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_sum64(v);
    __syncthreads();
    if (lane == 0)
        sh.warp64[warp] = v;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int w = 0; w < SC_WARPS; ++w)
        t += sh.warp64[w];
    return t;
}

// Rank 0 of a row's cluster: sh.list holds its n <= SC_THREADS candidates.
// Each candidate's place in the order and the masses before it come from a
// comparison with every other one (S threads share a candidate's), which for
// so few is shorter than a sort's or a bisection's barriers.
template <int S>
__device__ __noinline__ void pick_by_counting(const SampleArgs &a, int r, int n, int k, bool has_p, float p, float mp,
                                              float u, float m, float inv, u64 z_all)
{
    SampleShared &sh = sample_shared();
    const int i = threadIdx.x / S, part = threadIdx.x % S;
    const bool live = i < n;
    u64 *mass = sh.mass;
    const u64 x = live ? sh.list[i] : ~0ull;
    const float e = live ? expf((key_logit(~(uint32_t)(x >> 32)) - m) * inv) : 0.f;
    const u64 w = fixed_mass(e);
    // padded to whole steps (at most SC_THREADS / S places) with places behind all others, of no mass
    const int np = (n + 4 * S - 1) / (4 * S) * (4 * S);
    if (part == 0 && i < np) {
        mass[i] = w;
        if (!live)
            sh.list[i] = ~0ull;
    }
    __syncthreads();
    auto shared_sum = [&](u64 v) {
#pragma unroll
        for (int o = S / 2; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    u64 before = 0;
    uint32_t rank = 0;
    if (__any_sync(0xffffffffu, live)) {
        for (int j = 2 * part; j < np; j += 4 * S) {
            const ulonglong2 l0 = *reinterpret_cast<const ulonglong2 *>(&sh.list[j]);
            const ulonglong2 l1 = *reinterpret_cast<const ulonglong2 *>(&sh.list[j + 2 * S]);
            const ulonglong2 m0 = *reinterpret_cast<const ulonglong2 *>(&mass[j]);
            const ulonglong2 m1 = *reinterpret_cast<const ulonglong2 *>(&mass[j + 2 * S]);
            rank += (uint32_t)(l0.x < x) + (uint32_t)(l0.y < x) + (uint32_t)(l1.x < x) + (uint32_t)(l1.y < x);
            before += (l0.x < x ? m0.x : 0) + (l0.y < x ? m0.y : 0) + (l1.x < x ? m1.x : 0) + (l1.y < x ? m1.y : 0);
        }
        before = shared_sum(before);
#pragma unroll
        for (int o = S / 2; o > 0; o >>= 1)
            rank += __shfl_xor_sync(0xffffffffu, rank, o);
    }
    const bool top = live && (k <= 0 || rank < (uint32_t)k);
    u64 need = ~0ull;
    if (has_p) {
        const u64 zk = k > 0 ? block_sum64(top && part == 0 ? w : 0, sh) : z_all;
        need = needed_mass(p, zk);
    }
    const bool keep = top && (rank == 0 || (before < need && e >= mp));
    const u64 z = block_sum64(keep && part == 0 ? w : 0, sh);  // (its barriers: all have read mass[])
    if (live && part == 0)
        mass[i] = keep ? w : 0;
    __syncthreads();
    const u64 goal = goal_mass(u, z);
    if (!__any_sync(0xffffffffu, keep))
        return;
    const uint32_t idx = (uint32_t)x;
    before = 0;
    for (int j = 2 * part; j < np; j += 4 * S) {
        const ulonglong2 l0 = *reinterpret_cast<const ulonglong2 *>(&sh.list[j]);
        const ulonglong2 l1 = *reinterpret_cast<const ulonglong2 *>(&sh.list[j + 2 * S]);
        const ulonglong2 m0 = *reinterpret_cast<const ulonglong2 *>(&mass[j]);
        const ulonglong2 m1 = *reinterpret_cast<const ulonglong2 *>(&mass[j + 2 * S]);
        before += ((uint32_t)l0.x < idx ? m0.x : 0) + ((uint32_t)l0.y < idx ? m0.y : 0) +
                  ((uint32_t)l1.x < idx ? m1.x : 0) + ((uint32_t)l1.y < idx ? m1.y : 0);
    }
    before = shared_sum(before);
    if (keep && part == 0 && before <= goal && goal < before + w) {
        a.tokens[r] = (int)idx;
        if (a.probs)
            a.probs[r] = share(e, z);
    }
}

// Sums of N values over the block, to all threads; `turn` alternates the buffers.
template <int N>
__device__ __forceinline__ void block_sums(u64 (&v)[N], SampleShared &sh, int &turn)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, set = turn++ & 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = warp_sum64(v[i]);
        if (lane == 0)
            sh.x64[set][i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        u64 t = 0;
#pragma unroll
        for (int w = 0; w < SC_WARPS; ++w)
            t += sh.x64[set][i][w];
        v[i] = t;
    }
}

// The same for up to SC_LIST candidates, a few in each thread's registers:
// the cut's key, the last kept tie's index and the token's index by
// bisection, two bits a step.
__device__ __noinline__ void pick_by_bisection(const SampleArgs &a, int r, int n, int k, bool has_p, float p, float mp,
                                               float u, float m, float inv, u64 z_all)
{
    SampleShared &sh = sample_shared();
    constexpr int PER = SC_LIST / SC_THREADS;
    const int tid = threadIdx.x;
    uint32_t key[PER], idx[PER];
    float e[PER];
    u64 w[PER];
    uint32_t least = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = tid + i * SC_THREADS;
        const u64 x = at < n ? sh.list[at] : ~0ull;
        key[i] = ~(uint32_t)(x >> 32);  // (0, below every token's, where there is none)
        idx[i] = (uint32_t)x;
        e[i] = at < n ? expf((key_logit(key[i]) - m) * inv) : 0.f;
        w[i] = fixed_mass(e[i]);
        if (at < n)
            least = min(least, key[i]);
    }
    __syncthreads();
    int turn = 0;
    least = __reduce_min_sync(0xffffffffu, least);
    if ((tid & 31) == 0)
        sh.warp32[tid >> 5] = least;
    __syncthreads();
    for (int v = 0; v < SC_WARPS; ++v)
        least = min(least, sh.warp32[v]);
    // the keys differ in their bits below `top` only
    const uint32_t most = order_key(m);
    const int top = least == most ? 0 : (33 - __clz(least ^ most)) / 2 * 2;
    const uint32_t common = top >= 32 ? 0u : most >> top << top;
    uint32_t cut = 0;
    u64 ties = ~0ull, over = 0;  // ties of the cut that are kept; mass above it
    if (k > 0 && k < n) {
        uint32_t lo = common;
        u64 more = 0;  // tokens above the cut
        for (int bit = top - 2; bit >= 0; bit -= 2) {
            const uint32_t one = 1u << bit;
            u64 c[2] = {};
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                c[0] += (u64)(key[i] >= lo + one) | (u64)(key[i] >= lo + 2 * one) << 32;
                c[1] += key[i] >= lo + 3 * one;
            }
            block_sums(c, sh, turn);
            const u64 q[3] = {c[0] & 0xffffffffu, c[0] >> 32, c[1]};
            const int up = q[2] >= (u64)k ? 3 : q[1] >= (u64)k ? 2 : q[0] >= (u64)k ? 1 : 0;
            lo += up * one;
            if (up < 3)
                more = q[up];
        }
        cut = lo;
        ties = (u64)k - more;
    }
    if (has_p) {
        u64 c[1] = {};
#pragma unroll
        for (int i = 0; i < PER; ++i)
            c[0] += key[i] > cut ? w[i] : 0;
        block_sums(c, sh, turn);
        const u64 w_cut = cut ? fixed_mass(expf((key_logit(cut) - m) * inv)) : 0;
        const u64 zk = k > 0 ? c[0] + (cut ? ties * w_cut : 0) : z_all;
        const u64 need = needed_mass(p, zk);
        if (c[0] >= need) {
            uint32_t lo = common;
            for (int bit = top - 2; bit >= 0; bit -= 2) {
                const uint32_t one = 1u << bit;
                u64 f[3] = {};
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const u64 x = key[i] > cut ? w[i] : 0;
                    f[0] += key[i] >= lo + one ? x : 0;
                    f[1] += key[i] >= lo + 2 * one ? x : 0;
                    f[2] += key[i] >= lo + 3 * one ? x : 0;
                }
                block_sums(f, sh, turn);
                const int up = f[2] >= need ? 3 : f[1] >= need ? 2 : f[0] >= need ? 1 : 0;
                lo += up * one;
                if (up < 3)
                    over = f[up];
            }
            cut = lo;
            const u64 x = fixed_mass(expf((key_logit(cut) - m) * inv));
            ties = x > 0 ? (need - over + x - 1) / x : 1;
        } else if (cut && w_cut > 0) {
            ties = min(ties, (need - c[0] + w_cut - 1) / w_cut);
        }
    }
    // the least index at which a running sum over the tokens, by index, exceeds `goal`
    auto at_index = [&](const u64 (&x)[PER], u64 goal) {
        uint32_t lo = 0;
        for (int bit = 20; bit >= 0; bit -= 2) {  // (an index has at most 20 bits)
            const uint32_t one = 1u << bit;
            u64 f[3] = {};
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                f[0] += idx[i] < lo + one ? x[i] : 0;
                f[1] += idx[i] < lo + 2 * one ? x[i] : 0;
                f[2] += idx[i] < lo + 3 * one ? x[i] : 0;
            }
            block_sums(f, sh, turn);
            lo += (f[2] <= goal ? 3u : f[1] <= goal ? 2u : f[0] <= goal ? 1u : 0u) * one;
        }
        return lo;
    };
    uint32_t last_tie = 0xffffffffu;
    if (ties != ~0ull) {
        u64 t[PER], c[1] = {};
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            t[i] = key[i] == cut;
            c[0] += t[i];
        }
        block_sums(c, sh, turn);
        if (c[0] > ties)
            last_tie = at_index(t, ties - 1);
    }
    u64 z[1] = {};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool keep = key[i] > cut || (key[i] == cut && idx[i] <= last_tie);
        if (!keep || (e[i] < mp && key[i] != most))
            w[i] = 0;
        z[0] += w[i];
    }
    block_sums(z, sh, turn);
    const u64 goal = goal_mass(u, z[0]);
    const uint32_t token = at_index(w, goal);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (w[i] > 0 && idx[i] == token) {
            a.tokens[r] = (int)token;
            if (a.probs)
                a.probs[r] = share(e[i], z[0]);
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
    SampleShared &sh = sample_shared();
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
    // the row's settings are on their way with its logits
    const float tau = a.tau ? a.tau[r] : 1.f;
    const int k = a.top_k ? a.top_k[r] : 0;
    const float p = a.top_p ? a.top_p[r] : 1.f;
    const float mp_given = a.min_p ? a.min_p[r] : 0.f;
    const float u = a.u[r];

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
    const bool has_k = k > 0 && k < V;
    uint32_t k_key = 0;  // an order key that at least k tokens reach
    {
        const uint32_t mine = order_key(my_max);
        const int want = (k + C - 1) / C;
        if (has_k && want <= SC_THREADS) {
            // At least k / C (rounded up) of this CTA's tokens reach the threads' maximum of that rank, so at least k
            // of all reach the least of the CTAs' ones.  Two bits a step: the threads that reach each of three
            // thresholds, counted in ten bits each (the lower bits make little difference).
            for (int bit = 30; bit >= 14; bit -= 2) {
                const uint32_t t = k_key | (1u << bit);
                uint32_t n = (uint32_t)(mine >= t) | (uint32_t)(mine >= t + (1u << bit)) << 10 |
                             (uint32_t)(mine >= t + (2u << bit)) << 20;
                n = __reduce_add_sync(0xffffffffu, n);
                uint32_t *packed = sh.packed[(bit >> 1) & 1];
                if (lane == 0)
                    packed[warp] = n;
                __syncthreads();
                n = __reduce_add_sync(0xffffffffu, lane < SC_WARPS ? packed[lane] : 0u);
                k_key += ((n >> 20) >= (uint32_t)want ? 3u : ((n >> 10) & 1023u) >= (uint32_t)want ? 2u
                          : (n & 1023u) >= (uint32_t)want                                         ? 1u
                                                                                                  : 0u)
                         << bit;
            }
        }
        uint32_t top = __reduce_max_sync(0xffffffffu, mine);
        if (lane == 0)
            sh.warp32[warp] = top;
        __syncthreads();
        if (C > 1)
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (warp == 0) {
            top = __reduce_max_sync(0xffffffffu, lane < SC_WARPS ? sh.warp32[lane] : 0u);
            if (lane < C)
                st_cluster(&sh.x64[1][7][rank], (uint32_t)lane, (u64)top << 32 | k_key);
        }
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
        top = 0;
        for (int q = 0; q < C; ++q) {
            top = max(top, (uint32_t)(sh.x64[1][7][q] >> 32));
            k_key = min(k_key, (uint32_t)sh.x64[1][7][q]);
        }
        m = key_logit(top);
    }
    if (m == -INFINITY) {
        if (rank == 0 && tid == 0) {
            a.tokens[r] = -1;
            if (a.probs)
                a.probs[r] = 0.f;
        }
        return;  // (the whole cluster; its last DSMEM access was before the barrier)
    }
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
    const bool inf_row = m == INFINITY;
    if (inf_row) {  // the tokens at +inf share the mass
        tmax = my_max == INFINITY ? 0.f : -INFINITY;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < E; ++j)
                x.set(v, j, x.at(v, j) == INFINITY ? 0.f : -INFINITY);
        m = 0.f;
    }
    const float mp = mp_given > 0.f ? fminf(mp_given, 1.f) : 0.f;
    const bool has_p = p < 1.f;
    auto e_of = [&](float l) { return expf((l - m) * inv); };           // of a single token
    auto e_fast = [&](float l) { return fast_exp2((l - m) * c2); };     // in sums over many
    // below this no token has e >= min_p (with room for the roundings)
    const float l_mp = mp > 0.f ? m + (logf(mp) - 1e-3f) * (1.f / inv) : -INFINITY;

    // ---- the bound and, where it is needed, the mass of all
    float bound = -INFINITY;
    u64 z_all = 0;
    bool listed = false;  // the candidates fit the list
    if (has_k) {
        // (with m = inf its tokens alone have mass; a key below -inf's is no float)
        bound = inf_row || k_key <= order_key(-INFINITY) ? -INFINITY : key_logit(k_key);
        if (!has_p)
            bound = fmaxf(bound, l_mp);
        listed = true;
    } else if (has_p) {
        const float b0 = m - 8.f / c2, b1 = m - 14.f / c2, b2 = m - 20.f / c2;
        u64 s[1 + SC_TRIALS] = {};  // the mass, and that above each bound
        float t0 = 0.f, t1 = 0.f, t2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float l = x.at(v, j), e = e_fast(l);
                t += e;
                t0 += l >= b0 ? e : 0.f;
                t1 += l >= b1 ? e : 0.f;
                t2 += l >= b2 ? e : 0.f;
            }
            s[0] += fixed_mass(t);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            t0 += __shfl_xor_sync(0xffffffffu, t0, o);
            t1 += __shfl_xor_sync(0xffffffffu, t1, o);
            t2 += __shfl_xor_sync(0xffffffffu, t2, o);
        }
        s[0] = warp_sum64(s[0]);
        s[1] = fixed_mass(t0);
        s[2] = fixed_mass(t1);
        s[3] = fixed_mass(t2);
        cluster_sums<true>(s, sh, turn, C, rank);
        z_all = s[0];
        // (the trial masses are good to 1e-6; a bound that only just suffices is passed over)
        const u64 need = needed_mass(p, z_all), more = need + (need >> 16);
        const float b[SC_TRIALS] = {b0, b1, b2};
        for (int i = SC_TRIALS - 1; i >= 0; --i)
            if (s[1 + i] >= more) {
                bound = b[i];
                listed = true;  // (unless they are too many, as it turns out)
            }
        if (mp > 0.f)
            listed = true;  // as far as min_p goes
        bound = fmaxf(bound, l_mp);
    }

    // ---- the candidates at or above the bound, to rank 0
    if (listed) {
        const int set = turn++ & 1;
        if (tid == 0)
            sh.count = 0;
        __syncthreads();
        const int room = SC_SLOTS / C;
        if (tmax >= bound)  // (few threads hold a candidate)
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float l = x.at(v, j);
                    if (l >= bound && l > -INFINITY) {
                        const uint32_t at = atomicAdd(&sh.count, 1u);
                        if (at < (uint32_t)room)
                            st_cluster(&sh.slots[rank * room + at], 0u,
                                       ((u64)~order_key(l) << 32) | (uint32_t)index(v, j));
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
        bool fits = true;
        for (int q = 0; q < C; ++q) {
            n_all += sh.x64[set][0][q];
            fits = fits && sh.x64[set][0][q] <= (u64)room;
        }
        if (fits && n_all <= SC_LIST) {
            if (rank != 0)
                return;
            // in a row: a warp per CTA's share
            if (warp < C) {
                int at = 0;
                for (int q = 0; q < warp; ++q)
                    at += (int)sh.x64[set][0][q];
                const int nq = (int)sh.x64[set][0][warp];
                for (int i = lane; i < nq; i += 32)
                    sh.list[at + i] = sh.slots[warp * room + i];
            }
            __syncthreads();
            const int n = (int)n_all, kk = has_k ? k : 0;
            if (n <= SC_THREADS / 8)
                pick_by_counting<8>(a, r, n, kk, has_p, p, mp, u, m, inv, z_all);
            else if (n <= SC_THREADS / 2)
                pick_by_counting<2>(a, r, n, kk, has_p, p, mp, u, m, inv, z_all);
            else if (n <= SC_THREADS)
                pick_by_counting<1>(a, r, n, kk, has_p, p, mp, u, m, inv, z_all);
            else
                pick_by_bisection(a, r, n, kk, has_p, p, mp, u, m, inv, z_all);
            return;
        }
    }

    // ---- too many candidates, or no bound at all: the cut by bisection over the registers
    uint32_t cut = 0;    // order key of the last kept logit
    u64 ties = ~0ull;    // how many of the tokens that equal it are kept, by index
    u64 above = 0;       // mass of the tokens above it
    auto key_at = [&](int v, int j) { return order_key(x.at(v, j)); };
    // the logit from which on a token's key is at least t (keys below -inf's and above inf's are no floats)
    auto threshold = [&](uint32_t t) { return t <= order_key(-INFINITY) ? -INFINITY : key_logit(t); };
    if (has_k) {
        uint32_t lo = 0;  // the largest key with at least k tokens at or above
        for (int bit = 30; bit >= (E == 8 ? 16 : 0); bit -= 2) {  // two bits a step
            const uint32_t one = 1u << bit;
            const float f0 = threshold(lo + one), f1 = threshold(lo + 2 * one), f2 = threshold(lo + 3 * one);
            uint32_t n0 = 0, n1 = 0, n2 = 0;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float l = x.at(v, j);
                    n0 += l >= f0;
                    n1 += l >= f1;
                    n2 += l >= f2;
                }
            n0 = __reduce_add_sync(0xffffffffu, n0);
            n1 = __reduce_add_sync(0xffffffffu, n1);
            n2 = __reduce_add_sync(0xffffffffu, n2);
            u64 s[1] = {(u64)n0 | (u64)n1 << 21 | (u64)n2 << 42};
            cluster_sums<true>(s, sh, turn, C, rank);
            const uint32_t q0 = s[0] & 0x1fffffu, q1 = (s[0] >> 21) & 0x1fffffu, q2 = s[0] >> 42;
            lo += one * (q2 >= (uint32_t)k ? 3u : q1 >= (uint32_t)k ? 2u : q0 >= (uint32_t)k ? 1u : 0u);
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
        cluster_sums<false>(s, sh, turn, C, rank);
        above = s[0];
        ties = min(s[2], (u64)k - s[1]);
    }
    const u64 w_cut = cut ? fixed_mass(e_of(key_logit(cut))) : 0;
    if (has_p) {
        const u64 zk = has_k ? above + ties * w_cut : z_all;
        const u64 need = needed_mass(p, zk);
        if (above >= need || !has_k) {  // the cut moves up: the largest key with at least `need` at or above
            uint32_t lo = 0;
            u64 over = 0;  // mass above it
            const float cut_l = cut ? key_logit(cut) : -INFINITY;  // (a token at -inf has no mass)
            for (int bit = 30; bit >= (E == 8 ? 16 : 0); bit -= 2) {  // two bits a step
                const uint32_t one = 1u << bit;
                const float f0 = threshold(lo + one), f1 = threshold(lo + 2 * one), f2 = threshold(lo + 3 * one);
                u64 s[3] = {};
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float t0 = 0.f, t1 = 0.f, t2 = 0.f;
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        const float l = x.at(v, j), e = l > cut_l ? e_fast(l) : 0.f;
                        t0 += l >= f0 ? e : 0.f;
                        t1 += l >= f1 ? e : 0.f;
                        t2 += l >= f2 ? e : 0.f;
                    }
                    s[0] += fixed_mass(t0);
                    s[1] += fixed_mass(t1);
                    s[2] += fixed_mass(t2);
                }
                cluster_sums<false>(s, sh, turn, C, rank);
                const uint32_t up = s[2] >= need ? 3u : s[1] >= need ? 2u : s[0] >= need ? 1u : 0u;
                lo += up * one;
                if (up < 3)
                    over = s[up];  // the least threshold that falls short
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
        cluster_sums<false>(s, sh, turn, C, rank);
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
    const u64 goal = goal_mass(u, z);
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
                const float want = __ull2float_rz(goal - at) * 0x1p-40f;
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
                    a.probs[r] = share(pe, z);
                done = true;
            }
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
}

template <typename T, int NV>
cudaError_t launch_cluster(const SampleArgs &a, int T_rows, int C, int per_warp, cudaStream_t st)
{
    static thread_local int attr_dev = -1;  // per host thread
    int dev = 0;
    cudaGetDevice(&dev);
    if (attr_dev != dev) {
        cudaError_t e = cudaFuncSetAttribute(k_sample<T, NV>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_sample<T, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)sizeof(SampleShared));
        if (e != cudaSuccess)
            return e;
        attr_dev = dev;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)T_rows * C, 1, 1);
    cfg.blockDim = dim3(SC_THREADS, 1, 1);
    cfg.dynamicSmemBytes = sizeof(SampleShared);
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
    // (a row may begin inside a vector)
    const bool aligned = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && (T_rows == 1 || a.stride % E == 0);
    const int vectors = (a.V + E - 1) / E + (aligned ? 0 : 1);
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
