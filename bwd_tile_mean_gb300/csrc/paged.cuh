// paged.cuh -- problem description and helpers shared by the paged-cache
// kernels (append, page selection, one-token attention). Internal.
#pragma once

#include <cmath>

#include "vsa.h"
#include "vsa_internal.h"

namespace vsa {

// A validated vsa_paged_desc, passed to kernels by value.
struct Paged {
    int dtype;
    int B, Hq, Hkv, G;             // G = Hq / Hkv query heads per key/value head
    int page, page_log2;
    int num_pages, max_pages;
    int max_len;                   // max_pages * page
    long long page_stride;         // elements between pages
    long long tok_stride, head_stride;  // elements between a page's tokens / heads
    const int *table, *lens;
    float scale;
};

constexpr int kD = 128;

// Sequence length, clamped into what the page table can hold.
__device__ __forceinline__ int paged_len(const Paged &p, int b) { return clampi(__ldg(p.lens + b), 0, p.max_len); }
// Page id of logical page j of sequence b, -1 when there is no such page.
__device__ __forceinline__ int paged_id(const Paged &p, int b, int j) {
    if (j < 0 || j >= p.max_pages) return -1;
    const int id = __ldg(p.table + (long long)b * p.max_pages + j);
    return id >= 0 && id < p.num_pages ? id : -1;
}

// Host: descriptor -> Paged. The device arrays are only needed by the calls
// that launch (need_arrays).
inline vsa_status to_paged(const vsa_paged_desc *d, Paged *p, bool need_arrays) {
    if (!d) return VSA_ERR_NULL;
    if (d->layout != VSA_LAYOUT_BSHD && d->layout != VSA_LAYOUT_BHSD) return VSA_ERR_LAYOUT;
    if (d->dtype != VSA_DTYPE_BF16 && d->dtype != VSA_DTYPE_FP16) return VSA_ERR_DTYPE;
    if (d->B < 1 || d->Hq < 1 || d->Hkv < 1 || d->Hq % d->Hkv != 0) return VSA_ERR_SHAPE;
    if (d->D != kD) return VSA_ERR_UNSUPPORTED;
    int lg = 0;
    while ((1 << lg) < d->page && lg < 9) ++lg;
    if (d->page < 16 || d->page > 256 || (1 << lg) != d->page) return VSA_ERR_UNSUPPORTED;
    if (d->num_pages < 1 || d->max_pages < 1) return VSA_ERR_SHAPE;
    if ((long long)d->max_pages * d->page > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    if ((long long)d->B * d->Hq > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    const long long dense = (long long)d->page * d->Hkv * kD;
    if (d->page_stride != 0 && (d->page_stride < dense || d->page_stride % 8 != 0)) return VSA_ERR_SHAPE;
    if (!(d->scale >= 0.f) || std::isinf(d->scale)) return VSA_ERR_SHAPE;
    if (need_arrays) {
        if (!d->page_table || !d->seq_lens) return VSA_ERR_NULL;
        if (((uintptr_t)d->page_table | (uintptr_t)d->seq_lens) & 3u) return VSA_ERR_LAYOUT;
    }
    p->dtype = d->dtype;
    p->B = d->B;
    p->Hq = d->Hq;
    p->Hkv = d->Hkv;
    p->G = d->Hq / d->Hkv;
    p->page = d->page;
    p->page_log2 = lg;
    p->num_pages = d->num_pages;
    p->max_pages = d->max_pages;
    p->max_len = d->max_pages * d->page;
    p->page_stride = d->page_stride ? d->page_stride : dense;
    p->tok_stride = d->layout == VSA_LAYOUT_BSHD ? (long long)d->Hkv * kD : kD;
    p->head_stride = d->layout == VSA_LAYOUT_BSHD ? kD : (long long)d->page * kD;
    p->table = d->page_table;
    p->lens = d->seq_lens;
    p->scale = d->scale > 0.f ? d->scale : 1.0f / std::sqrt((float)kD);
    return VSA_OK;
}

// Host: a token stride argument (0: dense). False when it is not usable.
inline bool token_stride(int64_t given, int heads, long long *out) {
    const long long dense = (long long)heads * kD;
    *out = given ? given : dense;
    return given == 0 || (given >= dense && given % 8 == 0);
}

// Kernels of the paged calls are launched so that the next one on the stream
// may start while this one drains: every CTA waits for the work before it
// with grid_wait() before it touches memory, and lets the launch after it
// go ahead with grid_go().
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename A>
inline cudaError_t launch_paged(void (*kernel)(A), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                                const A &args, cudaStream_t s) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, args);
}

// Workspace of vsa_paged_attn.
struct PagedWs {
    size_t seg;         // [segments] int4: where a segment's pieces are
    size_t ml;          // [slots, rows] float2: running maximum (log2 units) and sum
    size_t o;           // [slots, rows, 128] fp32 unnormalised partial outputs
    size_t total;
};
PagedWs paged_ws(const Paged &p);

}  // namespace vsa
