// Attention over the paged cache for a planned batch (lora_prefix_attention).
//
//     out = sum_j w_j v_j / sum_j w_j,   w_j = 2^(s_j - m),   s_j = q . k_j * scale / log 2
//
// over the group's prefix, then the request's own tokens up to the query
// itself.  One pass over the keys with a running maximum m and sum per row;
// a prefix's keys are read once for the rows of all of the group's requests.
//
//  * k_attn_narrow: tiles of 16 query rows (the heads that share a key/value
//    head, times the tokens) and 64 keys.  A producer warp brings the keys'
//    and values' pages in by TMA (a page of a head is one box of rows, in the
//    128-byte swizzle that makes the ldmatrix reads free of bank conflicts)
//    through a ring of stages; four warps take 16 keys of a tile each, with
//    running statistics of their own, so the loop holds no barrier between
//    them; their sums are joined at a piece's end.  Bound by the cache's
//    bytes: a tile of 16 KB of keys and as much of values costs each warp 16
//    + 32 small products.
//  * k_attn_wide (attn_wide.cu): tiles of 256 rows and 128 keys on the tensor
//    memory's matrix instructions, for prefixes of many requests and for
//    prefill chunks.
//  * k_attn_combine: joins each row's pieces (the key axis is cut over the
//    SMs, see attn.h) and rounds once.
#include <cstring>

#include "attn_core.cuh"

namespace tcl {

namespace {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// c (16 x 8) += a (16 x 16) b (16 x 8), bf16 in, fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- narrow

constexpr int NA_WARPS = 4;
constexpr int NA_CONSUMERS = NA_WARPS * 32;
constexpr int NA_THREADS = NA_CONSUMERS + 32;  // and the producer warp
constexpr int NA_RING_BYTES = 96 * 1024;       // two CTAs per SM

template <int D>
struct NaShape {
    static constexpr int SIDE = NA_KEYS * D * 2;  // bytes of a tile's keys (or values)
    static constexpr int STAGES = NA_RING_BYTES / (2 * SIDE);
    static constexpr int ACC = STAGES * 2 * SIDE;         // float [NA_ROWS][D + 4]
    static constexpr int ML = ACC + NA_ROWS * (D + 4) * 4;  // float2 [NA_WARPS][NA_ROWS]
    static constexpr int SMEM = ML + NA_WARPS * NA_ROWS * 8 + 1024;
};

// Shared-memory offset of the 16-byte chunk c (of D / 8) of a tile's key.
__device__ __forceinline__ uint32_t kv_chunk(int key, int c)
{
    return (uint32_t)((c >> 3) * NA_KEYS * 128 + key * 128 + (((c & 7) ^ (key & 7)) << 4));
}

template <int D>
__device__ void na_produce(const CUtensorMap &mk, const CUtensorMap &mv, const AttnPlanDev &p, int oob_row,
                           unsigned char *smem, uint64_t *full, uint64_t *empty, uint32_t *hide)
{
    typedef NaShape<D> S;
    const int lane = threadIdx.x & 31;
    int32_t *status = p.hdr + AH_STATUS;
    // lane -> (side, half of the head, box of the tile)
    const int br = min(p.page, ATTN_BOX_MAX), nb = NA_KEYS / br;
    const int box = lane % nb, half = (lane / nb) % (D / 64), side = lane / (nb * (D / 64));
    const bool mine = side < 2;
    const CUtensorMap *map = side == 0 ? &mk : &mv;
    int it = 0;
    bool ok = true;
    PieceWalk w(p, AC_NARROW, blockIdx.x);
    while (ok && w.next(p.hkv)) {
        const int32_t *pages = pages_of(p, w.g.src);
        const int nkeys = w.g.nkeys;
        int key = w.tile0 * NA_KEYS + box * br;
        int page = mine && key < nkeys ? pages[key >> p.page_log2] : -1;
        for (int k = 0; k < w.ntiles; ++k, ++it) {
            const int s = it % S::STAGES, nkey = key + NA_KEYS;
            // the next tile's page id is on its way while this stage is waited for
            const int npage = mine && k + 1 < w.ntiles && nkey < nkeys ? pages[nkey >> p.page_log2] : -1;
            if (it >= S::STAGES && !mbar_wait_bounded(&empty[s], ((it / S::STAGES) - 1) & 1, status)) {
                ok = false;
                break;
            }
            const bool live = mine && key < nkeys;
            const unsigned lives = __ballot_sync(0xffffffffu, live);
            const unsigned bad = __ballot_sync(0xffffffffu, live && side == 0 && half == 0 && page < 0);
            if (lane == 0) {
                hide[s] = bad;  // bit = box, of lanes 0 .. nb - 1
                mbar_arrive_expect_tx(&full[s], (uint32_t)__popc(lives) * br * 128);
            }
            __syncwarp();
            if (live) {
                const int row = page < 0 ? oob_row : (page * p.hkv + w.h) * p.page + (key & (p.page - 1));
                tma_load_2d(smem + s * 2 * S::SIDE + side * S::SIDE + half * NA_KEYS * 128 + box * br * 128, map,
                            half * 64, row, &full[s]);
            }
            key = nkey;
            page = npage;
        }
    }
    // every load has landed before the CTA can exit
    for (int i = max(0, it - S::STAGES); i < it && ok; ++i)
        ok = mbar_wait_bounded(&full[i % S::STAGES], (i / S::STAGES) & 1, status);
}

__device__ __forceinline__ void na_bar() { asm volatile("bar.sync 1, %0;" ::"n"(NA_CONSUMERS) : "memory"); }

template <int D>
__global__ void __launch_bounds__(NA_THREADS, NA_CTAS_PER_SM)
    k_attn_narrow(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const AttnPlanDev p, const AttnArgs a, const bool after_wide)
{
    typedef NaShape<D> S;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[S::STAGES], empty[S::STAGES];
    __shared__ uint32_t hide[S::STAGES];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], NA_WARPS);
        }
        fence_mbar_init();
    }
    __syncthreads();
    // the plan, q and the cache; the partial rows' last reader.  After the wide kernel all of it is there: each of
    // its CTAs let this kernel start only once it had waited itself.  The two work side by side, and this one
    // ends after it, so that the combine kernel's wait covers both.
    if (!after_wide)
        pdl_wait();
    pdl_launch_dependents();
    if (warp == NA_WARPS) {
        na_produce<D>(mk, mv, p, a.oob_row, smem, full, empty, hide);
        if (after_wide)
            pdl_wait();
        return;
    }
    int32_t *status = p.hdr + AH_STATUS;
    float *acc_s = reinterpret_cast<float *>(smem + S::ACC);
    float2 *ml_s = reinterpret_cast<float2 *>(smem + S::ML);
    const int G = p.hq / p.hkv;
    const int r0 = lane >> 2, r1 = r0 + 8, c2 = (lane & 3) * 2;
    const int bshift = p.page >= 64 ? 6 : p.page == 32 ? 5 : 4;
    const uint32_t ring = smem_u32(smem);
    int it = 0;
    bool ok = true;  // no wait has run out
    PieceWalk w(p, AC_NARROW, blockIdx.x);
    while (w.next(p.hkv)) {
        const AttnSeg &g = w.g;
        // the rows' queries, in the product's operand layout
        uint32_t qa[D / 16][4];
        int lim0 = 0, lim1 = 0;
        const __nv_bfloat16 *q0 = nullptr, *q1 = nullptr;
        if (r0 < g.nrows) {
            const int gr = g.row0 + r0, t = gr / G;
            q0 = a.q + t * a.q_stride + (long long)(w.h * G + gr % G) * D + c2;
            lim0 = min(g.nkeys, max(0, t + g.lim));
        }
        if (r1 < g.nrows) {
            const int gr = g.row0 + r1, t = gr / G;
            q1 = a.q + t * a.q_stride + (long long)(w.h * G + gr % G) * D + c2;
            lim1 = min(g.nkeys, max(0, t + g.lim));
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            qa[k][0] = q0 ? *reinterpret_cast<const uint32_t *>(q0 + k * 16) : 0u;
            qa[k][1] = q1 ? *reinterpret_cast<const uint32_t *>(q1 + k * 16) : 0u;
            qa[k][2] = q0 ? *reinterpret_cast<const uint32_t *>(q0 + k * 16 + 8) : 0u;
            qa[k][3] = q1 ? *reinterpret_cast<const uint32_t *>(q1 + k * 16 + 8) : 0u;
        }
        const int lim_first = __shfl_sync(0xffffffffu, lim0, 0);  // of row 0: the smallest
        float acc[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        for (int k = 0; k < w.ntiles; ++k, ++it) {
            const int s = it % S::STAGES;
            ok = ok && mbar_wait_bounded(&full[s], (it / S::STAGES) & 1, status);
            const int key0 = (w.tile0 + k) * NA_KEYS + warp * 16;
            if (ok && key0 < g.nkeys && !((hide[s] >> ((warp * 16) >> bshift)) & 1u)) {
                const uint32_t kb = ring + s * 2 * S::SIDE, vb = kb + S::SIDE;
                float sc[2][4] = {};
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t b[4];
                    ldsm4(b, kb + kv_chunk(warp * 16 + (lane >> 4) * 8 + (lane & 7), kk * 2 + ((lane >> 3) & 1)));
                    mma16816(sc[0], qa[kk], b[0], b[1]);
                    mma16816(sc[1], qa[kk], b[2], b[3]);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = key0 + n * 8 + c2 + e;
                        sc[n][e] = key < lim0 ? sc[n][e] * a.scale_log2 : -INFINITY;
                        sc[n][2 + e] = key < lim1 ? sc[n][2 + e] * a.scale_log2 : -INFINITY;
                    }
                float x0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
                float x1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(m0, fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)));
                x1 = fmaxf(m1, fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)));
                const float b0 = x0 == -INFINITY ? 0.f : x0, b1 = x1 == -INFINITY ? 0.f : x1;
                const float f0 = pow2(m0 - b0), f1 = pow2(m1 - b1);
                if (__any_sync(0xffffffffu, x0 != m0 || x1 != m1)) {
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        acc[i][0] *= f0;
                        acc[i][1] *= f0;
                        acc[i][2] *= f1;
                        acc[i][3] *= f1;
                    }
                    l0 *= f0;
                    l1 *= f1;
                    m0 = x0;
                    m1 = x1;
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    sc[n][0] = pow2(sc[n][0] - b0);
                    sc[n][1] = pow2(sc[n][1] - b0);
                    sc[n][2] = pow2(sc[n][2] - b1);
                    sc[n][3] = pow2(sc[n][3] - b1);
                    l0 += sc[n][0] + sc[n][1];
                    l1 += sc[n][2] + sc[n][3];
                }
                // the weights in two bf16 parts (their sum is good to 16 bits): the products have time to spare
                const uint32_t ah[4] = {pack_bf16(sc[0][0], sc[0][1]), pack_bf16(sc[0][2], sc[0][3]),
                                        pack_bf16(sc[1][0], sc[1][1]), pack_bf16(sc[1][2], sc[1][3])};
                const uint32_t al[4] = {pack_bf16(sc[0][0] - bf16lo(ah[0]), sc[0][1] - bf16hi(ah[0])),
                                        pack_bf16(sc[0][2] - bf16lo(ah[1]), sc[0][3] - bf16hi(ah[1])),
                                        pack_bf16(sc[1][0] - bf16lo(ah[2]), sc[1][1] - bf16hi(ah[2])),
                                        pack_bf16(sc[1][2] - bf16lo(ah[3]), sc[1][3] - bf16hi(ah[3]))};
                bool wrote = false;
                // values that no row sees (beyond the keys) count as 0, whatever they hold
                if (key0 + 16 > g.nkeys) {
                    for (int i = lane; i < 16 * (D / 8); i += 32) {
                        const int key = i / (D / 8);
                        if (key0 + key >= g.nkeys)
                            *reinterpret_cast<uint4 *>(smem + s * 2 * S::SIDE + S::SIDE +
                                                       kv_chunk(warp * 16 + key, i % (D / 8))) = make_uint4(0, 0, 0, 0);
                    }
                    wrote = true;
                    __syncwarp();
                }
                // values that some rows do not see: one that is not finite would reach them as 0 * inf.  Such
                // keys are taken out of the product and added row by row.
                if (key0 + 16 > lim_first) {
                    unsigned odd = 0;
                    for (int i = lane; i < 16 * (D / 8); i += 32) {
                        const uint4 x = lds128(smem + s * 2 * S::SIDE + S::SIDE +
                                               kv_chunk(warp * 16 + i / (D / 8), i % (D / 8)));
                        if (bf16_pair_not_finite(x.x) || bf16_pair_not_finite(x.y) || bf16_pair_not_finite(x.z) ||
                            bf16_pair_not_finite(x.w))
                            odd |= 1u << (i / (D / 8));
                    }
                    odd = __reduce_or_sync(0xffffffffu, odd);
                    for (unsigned left = odd; left; left &= left - 1) {
                        const int key = __ffs(left) - 1, src = (lane & ~3) | ((key & 7) >> 1), e = key & 1;
                        const float p0 = __shfl_sync(0xffffffffu, e ? (key & 8 ? sc[1][1] : sc[0][1])
                                                                    : (key & 8 ? sc[1][0] : sc[0][0]), src);
                        const float p1 = __shfl_sync(0xffffffffu, e ? (key & 8 ? sc[1][3] : sc[0][3])
                                                                    : (key & 8 ? sc[1][2] : sc[0][2]), src);
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            const uint32_t v = *reinterpret_cast<const uint32_t *>(
                                smem + s * 2 * S::SIDE + S::SIDE + kv_chunk(warp * 16 + key, i) + c2 * 2);
                            if (key0 + key < lim0) {
                                acc[i][0] += p0 * bf16lo(v);
                                acc[i][1] += p0 * bf16hi(v);
                            }
                            if (key0 + key < lim1) {
                                acc[i][2] += p1 * bf16lo(v);
                                acc[i][3] += p1 * bf16hi(v);
                            }
                        }
                        __syncwarp();
                        for (int i = lane; i < D / 8; i += 32)
                            *reinterpret_cast<uint4 *>(smem + s * 2 * S::SIDE + S::SIDE +
                                                       kv_chunk(warp * 16 + key, i)) = make_uint4(0, 0, 0, 0);
                        wrote = true;
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int dd = 0; dd < D / 16; ++dd) {
                    uint32_t b[4];
                    ldsm4t(b, vb + kv_chunk(warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), dd * 2 + (lane >> 4)));
                    mma16816(acc[2 * dd], ah, b[0], b[1]);
                    mma16816(acc[2 * dd + 1], ah, b[2], b[3]);
                    mma16816(acc[2 * dd], al, b[0], b[1]);
                    mma16816(acc[2 * dd + 1], al, b[2], b[3]);
                }
                if (wrote)
                    fence_proxy_async_smem();  // before the stage's next TMA write
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&empty[s]);
        }

        // the four warps' sums on a common maximum, in warp order
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if ((lane & 3) == 0) {
            ml_s[warp * NA_ROWS + r0] = make_float2(m0, l0);
            ml_s[warp * NA_ROWS + r1] = make_float2(m1, l1);
        }
        na_bar();
        float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
        for (int v = 0; v < NA_WARPS; ++v) {
            M0 = fmaxf(M0, ml_s[v * NA_ROWS + r0].x);
            M1 = fmaxf(M1, ml_s[v * NA_ROWS + r1].x);
        }
        const float f0 = pow2(m0 - (M0 == -INFINITY ? 0.f : M0)), f1 = pow2(m1 - (M1 == -INFINITY ? 0.f : M1));
        const long long out0 =
            (long long)blockIdx.x * NA_ROWS + g.rows0 + (long long)w.h * g.nrows;
        if (tid < g.nrows) {
            float M = -INFINITY, L = 0.f;
            for (int v = 0; v < NA_WARPS; ++v)
                M = fmaxf(M, ml_s[v * NA_ROWS + tid].x);
            for (int v = 0; v < NA_WARPS; ++v)
                L += ml_s[v * NA_ROWS + tid].y * pow2(ml_s[v * NA_ROWS + tid].x - (M == -INFINITY ? 0.f : M));
            p.part_ml[out0 + tid] = make_float2(M, L);
        }
        for (int v = 0; v < NA_WARPS; ++v) {
            if (warp == v) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    float2 *x0 = reinterpret_cast<float2 *>(acc_s + r0 * (D + 4) + i * 8 + c2);
                    float2 *x1 = reinterpret_cast<float2 *>(acc_s + r1 * (D + 4) + i * 8 + c2);
                    if (r0 < g.nrows) {
                        const float2 o = v ? *x0 : make_float2(0.f, 0.f);
                        *x0 = make_float2(o.x + acc[i][0] * f0, o.y + acc[i][1] * f0);
                    }
                    if (r1 < g.nrows) {
                        const float2 o = v ? *x1 : make_float2(0.f, 0.f);
                        *x1 = make_float2(o.x + acc[i][2] * f1, o.y + acc[i][3] * f1);
                    }
                }
            }
            na_bar();
        }
        for (int i = tid; i < g.nrows * (D / 4); i += NA_CONSUMERS) {
            const int r = i / (D / 4), c = (i % (D / 4)) * 4;
            *reinterpret_cast<float4 *>(p.part + (out0 + r) * D + c) =
                *reinterpret_cast<const float4 *>(acc_s + r * (D + 4) + c);
        }
    }
}

// ---------------------------------------------------------------- combine

// A warp per (query token, head): its pieces of the prefix, then of the
// request's own tokens, in the order of the keys.
template <int D>
__global__ void __launch_bounds__(128) k_attn_combine(const AttnPlanDev p, const AttnArgs a)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = ((long long)blockIdx.x * 128 + threadIdx.x) >> 5;
    pdl_wait();
    pdl_launch_dependents();
    if (row >= (long long)a.TQ * p.hq)
        return;
    const int t = (int)(row / p.hq), hq = (int)(row % p.hq), G = p.hq / p.hkv, h = hq / G;
    const int b = p.tok_req[t];
    long long base[2] = {0, 0};
    int pitch[2] = {0, 0}, n[2] = {0, 0};
    if (b >= 0) {
        const int grp = p.grp[b];
        const int first[2] = {grp >= 0 ? p.pseg[grp] : -1, p.sseg[b]};
        const int t0[2] = {grp >= 0 ? p.g_row0[grp] : 0, p.q_off[b]};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (first[k] < 0)
                continue;
            const int cls = first[k] & 1, tr = cls == AC_WIDE ? WA_ROWS : NA_ROWS;
            const long long *len = p.len + cls * AL_WORDS;
            const int r = (t - t0[k]) * G + hq % G;
            const AttnSeg &g = p.seg[cls][(first[k] >> 1) + r / tr];
            if (g.ntiles == 0)
                continue;
            const long long a0 = g.a + (long long)h * g.ntiles, run = len[AL_RUN];
            const int c0 = (int)(a0 / run);
            n[k] = (int)((a0 + g.ntiles - 1) / run) - c0 + 1;
            pitch[k] = p.pitch[cls];
            base[k] = len[AL_PART] + (long long)c0 * pitch[k] + g.rows0 + (long long)h * g.nrows + r % tr;
        }
    }
    auto part_row = [&](int i) {
        return i < n[0] ? base[0] + (long long)i * pitch[0] : base[1] + (long long)(i - n[0]) * pitch[1];
    };
    const int np = n[0] + n[1];
    float M = -INFINITY;
    for (int i = lane; i < np; i += 32)
        M = fmaxf(M, p.part_ml[part_row(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float B = M == -INFINITY ? 0.f : M;
    float acc[E] = {}, L = 0.f;
#pragma unroll 4
    for (int i = 0; i < np; ++i) {
        const long long pr = part_row(i);
        const float2 ml = p.part_ml[pr];
        const float w = pow2(ml.x - B);
        L += w * ml.y;
        const float *x = p.part + pr * D + lane * E;
        if constexpr (E == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(x);
            acc[0] += w * v.x;
            acc[1] += w * v.y;
            acc[2] += w * v.z;
            acc[3] += w * v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(x);
            acc[0] += w * v.x;
            acc[1] += w * v.y;
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    __nv_bfloat16 *o = a.out + t * a.out_stride + (long long)hq * D + lane * E;
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(o) =
            make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(o) = pack_bf16(acc[0] * inv, acc[1] * inv);
    if (a.lse && lane == 0)
        a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.693147180559945f;
}

template <int D>
cudaError_t run_attn(const AttnPlanDev &p, const AttnArgs &a, const lora_kv_cache &cache, cudaStream_t st)
{
    static thread_local int attr_dev = -1;  // per host thread
    int dev = 0;
    cudaGetDevice(&dev);
    if (attr_dev != dev) {
        cudaError_t e = cudaFuncSetAttribute(k_attn_narrow<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             NaShape<D>::SMEM);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_attn_narrow<D>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess)
            return e;
        attr_dev = dev;
    }
    CUtensorMap mk, mv;
    std::memcpy(&mk, cache.map_k, sizeof(mk));
    std::memcpy(&mv, cache.map_v, sizeof(mv));
    // which classes there can be: a request's rows are its tokens times the heads that share a key/value head
    const int G = p.hq / p.hkv;
    const bool wide = (long long)a.TQ * G > NA_ROWS;
    const bool narrow = G <= NA_ROWS && (!wide || a.B > 1);
    cudaError_t e = cudaSuccess;
    if (wide)
        e = launch_attn_wide(p, a, mk, mv, cache.v, st);
    if (e == cudaSuccess && narrow)
        e = launch_pdl(k_attn_narrow<D>, dim3(p.ctas[AC_NARROW]), NA_THREADS, NaShape<D>::SMEM, st, mk, mv, p, a,
                       wide);
    if (e != cudaSuccess)
        return e;
    const long long rows = (long long)a.TQ * p.hq;
    return launch_pdl(k_attn_combine<D>, dim3((unsigned)((rows + 3) / 4)), 128, 0, st, p, a);
}

}  // namespace

cudaError_t launch_attn(const AttnPlanDev &p, const AttnArgs &a, const lora_kv_cache &cache, cudaStream_t st)
{
    return p.d == 64 ? run_attn<64>(p, a, cache, st) : run_attn<128>(p, a, cache, st);
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
    if (!q_dev || !out_dev || q_dev == out_dev || q_stride < row || out_stride < row || q_stride % 8 ||
        out_stride % 8 || ((reinterpret_cast<uintptr_t>(q_dev) | reinterpret_cast<uintptr_t>(out_dev)) & 15u))
        return LORA_ERR_INVALID_ARG;
    if (!cache->maps_ready)
        return LORA_ERR_CUDA;
    AttnArgs a{};
    a.q = static_cast<const __nv_bfloat16 *>(q_dev);
    a.out = static_cast<__nv_bfloat16 *>(out_dev);
    a.lse = lse_dev;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.TQ = plan->TQ;
    a.B = plan->B;
    a.oob_row = cache->num_pages * cache->hkv * cache->page_size;
    return launch_attn(p, a, *cache, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
