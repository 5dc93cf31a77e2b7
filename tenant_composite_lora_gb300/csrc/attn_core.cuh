// Device helpers shared by the attention kernels.
#pragma once

#include <cuda.h>

#include "attn.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace tcl {

__device__ __forceinline__ float pow2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ bool bf16_not_finite(uint32_t half) { return (half & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ bool bf16_pair_not_finite(uint32_t w)
{
    return bf16_not_finite(w) || bf16_not_finite(w >> 16);
}

// The pieces of a CTA's run over one class's sequence, in order.
struct PieceWalk {
    const AttnSeg *seg;
    long long p, p1;
    int s, h, tile0, ntiles;
    AttnSeg g;
    __device__ __forceinline__ PieceWalk(const AttnPlanDev &pl, int cls, int cta)
    {
        const long long run = pl.len[cls * AL_WORDS + AL_RUN], all = pl.len[cls * AL_WORDS + AL_TILES];
        seg = pl.seg[cls];
        p = cta * run;
        p1 = min(all, p + run);
        s = p < p1 ? pl.cta_seg[cls][cta] - 1 : 0;
        g.a = 0;
        g.ntiles = 0;
        ntiles = 0;
    }
    __device__ __forceinline__ bool next(int hkv)
    {
        p += ntiles;
        if (p >= p1)
            return false;
        while (p >= g.a + (long long)g.ntiles * hkv)
            g = seg[++s];
        const long long o = p - g.a;
        h = (int)(o / g.ntiles);
        tile0 = (int)(o - (long long)h * g.ntiles);
        ntiles = (int)min((long long)(g.ntiles - tile0), p1 - p);
        return true;
    }
};

__device__ __forceinline__ const int32_t *pages_of(const AttnPlanDev &p, int src)
{
    return src < 0 ? p.p_pages + (long long)~src * p.max_ppages : p.s_pages + (long long)src * p.max_spages;
}

// Launches with programmatic dependent launch: the kernel may start before
// the one before it on the stream has ended, and waits itself (pdl_wait).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace tcl
