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
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxHeads = 65536;  // key/value heads: a token's bytes stay within 32 bits

// Sequence length, clamped into what the page table can hold.
__device__ __forceinline__ int paged_len(const Paged &p, int b) { return clampi(p.lens[b], 0, p.max_len); }
// Page id of logical page j of sequence b, -1 when there is no such page.
__device__ __forceinline__ int paged_id(const Paged &p, int b, int j) {
    if (j < 0 || j >= p.max_pages) return -1;
    const int id = p.table[(long long)b * p.max_pages + j];
    return id >= 0 && id < p.num_pages ? id : -1;
}

// Host: descriptor -> Paged. The device arrays are only needed by the calls
// that launch (need_arrays).
inline vsa_status to_paged(const vsa_paged_desc *d, Paged *p, bool need_arrays) {
    if (!d) return VSA_ERR_NULL;
    if (d->layout != VSA_LAYOUT_BSHD && d->layout != VSA_LAYOUT_BHSD) return VSA_ERR_LAYOUT;
    if (d->dtype != VSA_DTYPE_BF16 && d->dtype != VSA_DTYPE_FP16) return VSA_ERR_DTYPE;
    if (d->B < 1 || d->Hq < 1 || d->Hkv < 1 || d->Hq % d->Hkv != 0) return VSA_ERR_SHAPE;
    if (d->D != kD || d->Hkv > kMaxHeads) return VSA_ERR_UNSUPPORTED;
    int lg = 0;
    while ((1 << lg) < d->page && lg < 9) ++lg;
    if (d->page < 16 || d->page > 256 || (1 << lg) != d->page) return VSA_ERR_UNSUPPORTED;
    if (d->num_pages < 1 || d->max_pages < 1) return VSA_ERR_SHAPE;
    if ((long long)d->max_pages * d->page > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    if ((long long)d->B * d->Hq > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    const long long dense = (long long)d->page * d->Hkv * kD;
    if (d->page_stride != 0 && (d->page_stride < dense || d->page_stride % 8 != 0)) return VSA_ERR_SHAPE;
    if (!(d->scale >= 0.f) || std::isinf(d->scale * kLog2e)) return VSA_ERR_SHAPE;
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

// x / d for 0 <= x: in 32 bits where they hold it.
__device__ __forceinline__ int div_small(long long x, int d) {
    return x <= 0x7fffffffLL ? (int)((unsigned)x / (unsigned)d) : (int)(x / d);
}

// Equal contiguous runs of the work of a list of entries, whatever their
// sizes: entry n has size_of(n) units (n < N), the units of all entries end
// to end are dealt to `workers` workers (at least min_per units each), and a
// CTA has `per_cta` neighbouring workers. Called by the whole CTA (W warps);
// every thread gets the CTA's run and the entry that holds its first unit.
struct Run {
    long long x0, x1, total, per;  // this CTA's units, all units, units per worker
    int n;                         // entry that holds x0 (x0 < x1)
    long long before;              // units of the entries before n
};
template <int W, typename F>
__device__ __forceinline__ Run find_run(int N, F size_of, int workers, int min_per, int per_cta) {
    __shared__ long long s_warp[W];
    __shared__ long long s_before;
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    auto size = [&](int n) -> long long { return n < N ? size_of(n) : 0; };
    if (tid == 0) s_n = 0, s_before = 0;
    // inclusive scan of one value per thread over the CTA; *all gets the sum
    auto scan = [&](long long v, long long *all) {
        long long inc = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += y;
        }
        if (lane == 31) s_warp[wid] = inc;
        __syncthreads();
        *all = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == wid) inc += *all;
            *all += s_warp[w];
        }
        return inc;
    };
    const long long v0 = size(tid);
    long long total, inc = scan(v0, &total);
    const long long inc0 = inc, all0 = total;
    for (int n0 = W * 32; n0 < N; n0 += W * 32) {
        long long all;
        __syncthreads();  // s_warp was read
        scan(size(n0 + tid), &all);
        total += all;
    }
    Run r;
    r.total = total;
    r.per = (total + workers - 1) / workers;
    if (r.per < min_per) r.per = min_per;
    r.x0 = (long long)blockIdx.x * r.per * per_cta;
    r.x1 = r.x0 + r.per * per_cta < total ? r.x0 + r.per * per_cta : total;
    r.n = 0;
    r.before = 0;
    if (r.x0 >= r.x1) return r;  // no work, for the whole CTA
    long long carry = 0, v = v0, all = all0;
    inc = inc0;
    for (int n0 = 0; n0 < N;) {
        inc += carry;
        if (inc - v <= r.x0 && r.x0 < inc) {  // one thread of the CTA
            s_n = n0 + tid;
            s_before = inc - v;
        }
        carry += all;
        n0 += W * 32;
        if (carry > r.x0 || n0 >= N) break;
        __syncthreads();  // s_warp was read
        v = size(n0 + tid);
        inc = scan(v, &all);
    }
    __syncthreads();
    r.n = s_n;
    r.before = s_before;
    return r;
}

// Kernels of the paged calls are launched so that the next one on the stream
// may start while this one drains: every CTA waits for the work before it
// with grid_wait() before it touches memory, and lets the launch after it go
// ahead with grid_go() when its streaming is over. What the work before may
// have written is read with ordinary loads: __ldg promises memory that no one
// writes while the kernel runs, its wait included, and could be moved before
// the wait. Measured (us, such launches
// / plain ones): one-token append 2.7 / 2.9, attention of 101 keys 3.7 / 4.1,
// select and attend 24.0 / 25.1. Letting the next launch in at the kernel's
// start instead takes slots from its own CTAs: 4 sequences of 8,000 pages
// 39 us for a selection against 32.
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
    const cudaError_t e = cudaLaunchKernelEx(&c, kernel, args);
    if (e != cudaSuccess) cudaGetLastError();  // returned to the caller, not left for the next launch
    return e;
}

// Workspace of vsa_page_select and vsa_paged_attn (each uses its own part).
struct PagedWs {
    size_t keys;        // [B * Hkv, max_pages] uint32 score keys
    size_t seg;         // [segments] int4: where a segment's pieces are
    size_t ml;          // [slots, rows] float4: maximum (log2 units), sum of weights, of rounded weights, 0
    size_t o;           // [slots, rows, 128] fp32 unnormalised partial outputs
    size_t total;
};
PagedWs paged_ws(const Paged &p);

}  // namespace vsa
