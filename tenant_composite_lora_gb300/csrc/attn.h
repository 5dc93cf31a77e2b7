// The attention step's objects and launchers (paged cache, plan), shared by
// their translation units.
#pragma once

#include "internal.h"

struct lora_kv_cache {
    int num_pages, page_size, hkv, d, device;
    __nv_bfloat16 *k, *v;  // [num_pages][hkv][page_size][d], the caller's
};

namespace tcl {

// Header words of a plan (device int32).
enum { AH_STATUS = 0, AH_NREQ = 1, AH_NGRP = 2, AH_TQ = 3, AH_WORDS = 16 };

// A plan on the device.  Lengths are already checked against their tables:
// a request's or group's length is 0 where it was malformed, a page is -1
// where its id was.
struct AttnPlanDev {
    int32_t *hdr;        // [AH_WORDS]
    int32_t *q_off;      // [max_requests + 1]
    int32_t *s_len;      // [max_requests]
    int32_t *grp;        // [max_requests] group of each request, -1: none
    int32_t *p_len;      // [max_groups]
    int32_t *tok_req;    // [max_queries] request of each query token, -1: none
    int32_t *s_pages;    // [max_requests][max_spages]
    int32_t *p_pages;    // [max_groups][max_ppages]
    int max_spages, max_ppages;
    int hq, hkv, d, page, page_log2;
};

struct AttnPlanSrc {
    const int32_t *q_off, *s_len, *s_pages, *g_off, *p_len, *p_pages;
    int s_stride, p_stride, B, NG, TQ, num_pages;
};

cudaError_t launch_attn_plan(const AttnPlanDev &p, const AttnPlanSrc &src, cudaStream_t st);

struct AttnArgs {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    float *lse;
    long long q_stride, out_stride;
    const __nv_bfloat16 *k, *v;
    float scale;
    int TQ;
};
cudaError_t launch_attn(const AttnPlanDev &p, const AttnArgs &a, cudaStream_t st);

}  // namespace tcl

struct lora_attn_plan {
    int max_requests, max_groups, max_queries, device;
    int TQ, num_pages;
    bool built;
    tcl::AttnPlanDev dev;
};
