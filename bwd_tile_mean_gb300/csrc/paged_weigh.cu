// paged_weigh.cu -- the attention weight that each page receives
// (vsa_paged_attn_weigh), and the eviction of the pages that received least
// (vsa_page_evict).
//
//   weight[b, h, j] = decay weight[b, h, j] + sum_(query heads of h) sum_(u in page j) P_u,
//   P_u = exp(scale q.k_u - LSE)
//
// The attention (paged_attn.cuh) walks each key once with a running maximum, so
// a key's P is known only when its row is finished. It leaves, per row and block
// of 16 keys, the sum of the block's exponentials and the maximum that they are
// relative to: 8 bytes per row and block against the block's 4 to 8 KB of keys
// and values. k_page_weigh puts them over the rows' LSE, per page.
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace vsa {
namespace {

struct WeighArgs {
    Paged p;
    const int *idx, *cnt;
    int cap;
    const float *lse;
    const float2 *bw;      // [segments, blocks, rows]
    int blocks, rows, rc;
    const float *in;       // [B, Hkv, max_pages]
    float *out;
    float decay, drop;     // drop: the attention's lift of P, undone
};
constexpr int kWeighThreads = 128;

// Sum of P over `n` blocks from entry block `blk` of list row bh, all of its query heads.
__device__ __forceinline__ float mass_of(const WeighArgs &a, long long bh, int blk, int n) {
    const Paged &p = a.p;
    const int b = (int)(bh / p.Hkv), h = (int)(bh % p.Hkv);
    const float *lse = a.lse + (long long)b * p.Hq + h * p.G;
    float mass = 0.f;
    for (int r = 0; r < a.rc; ++r) {
        const int rows = min(a.rows, p.G - r * a.rows);
        const float2 *w = a.bw + ((bh * a.rc + r) * a.blocks + blk) * a.rows;
        for (int i = 0; i < rows; ++i) {
            const float ref = lse[r * a.rows + i] * kLog2e;
            for (int k = 0; k < n; ++k) {
                const float2 x = w[k * a.rows + i];
                if (x.x != 0.f) mass += x.x * ptx::ex2(x.y - ref);
            }
        }
    }
    return mass * a.drop;
}
__device__ __forceinline__ float aged(const WeighArgs &a, long long at) { return a.decay == 0.f ? 0.f : a.decay * a.in[at]; }

// All pages: one thread per page.
__global__ void __launch_bounds__(kWeighThreads) k_page_weigh(WeighArgs a) {
    const Paged &p = a.p;
    const int chunks = (p.max_pages + kWeighThreads - 1) / kWeighThreads;
    const long long bh = blockIdx.x / chunks;
    const int j = (int)(blockIdx.x % chunks) * kWeighThreads + threadIdx.x;
    grid_wait();
    grid_go();
    if (j >= p.max_pages) return;
    const int len = paged_len(p, (int)(bh / p.Hkv)), from = j << p.page_log2;
    const long long at = bh * p.max_pages + j;
    if (from < len) {
        const int live = min(len - from, p.page);
        const float mass = mass_of(a, bh, from / 16, (live + 15) / 16);
        a.out[at] = a.decay == 0.f ? mass : fmaf(a.decay, a.in[at], mass);
    } else if (a.out != a.in) {
        a.out[at] = a.in[at];
    }
}

// Listed pages: one CTA per list. A list that is not ascending may name a page
// twice: its entries are then added one after another.
__global__ void __launch_bounds__(kWeighThreads) k_page_weigh_listed(WeighArgs a) {
    __shared__ float s_mass[kWeighThreads];
    const Paged &p = a.p;
    const long long bh = blockIdx.x;
    const int tid = threadIdx.x;
    grid_wait();
    grid_go();
    const int len = paged_len(p, (int)(bh / p.Hkv)), cnt = clampi(a.cnt[bh], 0, a.cap);
    const int *idx = a.idx + bh * a.cap;
    float *out = a.out + bh * p.max_pages;
    for (int j = tid; j < p.max_pages; j += kWeighThreads) {
        const long long at = bh * p.max_pages + j;
        if ((long long)j << p.page_log2 < len) {
            if (a.decay != 1.f || a.out != a.in) a.out[at] = aged(a, at);
        } else if (a.out != a.in) {
            a.out[at] = a.in[at];
        }
    }
    bool ascending = true;
    for (int n = tid + 1; n < cnt; n += kWeighThreads) ascending = ascending && idx[n - 1] < idx[n];
    ascending = __syncthreads_and(ascending);
    const int blocks = p.page / 16;
    for (int n0 = 0; n0 < cnt; n0 += kWeighThreads) {
        const int n = n0 + tid, j = n < cnt ? idx[n] : -1;
        const bool on = j >= 0 && j < p.max_pages && (long long)j << p.page_log2 < len;
        const float mass = on ? mass_of(a, bh, n * blocks, blocks) : 0.f;
        if (ascending) {
            if (on) out[j] += mass;
        } else {
            s_mass[tid] = mass;
            __syncthreads();
            if (tid == 0)
                for (int i = 0; i < kWeighThreads && n0 + i < cnt; ++i) {
                    const int at = idx[n0 + i];
                    if (at >= 0 && at < p.max_pages && (long long)at << p.page_log2 < len) out[at] += s_mass[i];
                }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- eviction

struct EvictArgs {
    Paged p;
    const float *weight;
    int keep, first, last, freed_cap;
    int *table_out, *lens_out;
    float *weight_out;
    int *freed, *cnt;
    uint32_t *keys;  // [B, max_pages] order-preserving keys of the pages' weights
    int *len;        // [B] the lengths: lens_out may be the lengths themselves
};
constexpr int kSumThreads = 256, kMoveThreads = 512, kMoveWarps = kMoveThreads / 32;

// A float's order as an unsigned's; NaN with -inf, -0 with 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Weights over the heads, as keys. The heads are added in fp64: the sum, rounded once to fp32, does not depend on an order.
__global__ void __launch_bounds__(kSumThreads) k_evict_sums(EvictArgs a) {
    const Paged &p = a.p;
    const int chunks = (p.max_pages + kSumThreads - 1) / kSumThreads;
    const int b = (int)(blockIdx.x / chunks), j = (int)(blockIdx.x % chunks) * kSumThreads + threadIdx.x;
    grid_wait();
    grid_go();
    const int raw = p.lens[b], len = clampi(raw, 0, p.max_len);
    if (j == 0) a.len[b] = raw;
    if (j >= p.max_pages || (long long)j << p.page_log2 >= len) return;
    const float *w = a.weight + (long long)b * p.Hkv * p.max_pages + j;
    double sum = 0.0;
#pragma unroll 8
    for (int h = 0; h < p.Hkv; ++h) sum += (double)w[(long long)h * p.max_pages];
    a.keys[(long long)b * p.max_pages + j] = order_key((float)sum);
}

// One CTA per row: sequence b's table (row 0 of Hkv + 1) or a head's weights. Each finds the last key to stay by itself,
// 8 bits at a time, then moves its row in ascending chunks: an entry moves to a place at or before its own, and a chunk
// is read before any of it is written, so the row may be moved in place.
__global__ void __launch_bounds__(kMoveThreads) k_evict_move(EvictArgs a) {
    __shared__ int s_hist[256];
    __shared__ int s_bin, s_left, s_warp[kMoveWarps];
    const Paged &p = a.p;
    const int b = (int)(blockIdx.x / (p.Hkv + 1)), row = (int)(blockIdx.x % (p.Hkv + 1)) - 1;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, P = p.max_pages;
    grid_wait();
    grid_go();
    const int raw = a.len[b], len = clampi(raw, 0, p.max_len), n = (len + p.page - 1) >> p.page_log2;
    const long long at = row < 0 ? (long long)b * P : ((long long)b * p.Hkv + row) * P;
    const int gone = n > a.keep ? n - a.keep : 0;
    if (row < 0) {
        for (int i = gone + tid; i < a.freed_cap; i += kMoveThreads) a.freed[(long long)b * a.freed_cap + i] = -1;
        if (tid == 0) {
            a.cnt[b] = gone;
            a.lens_out[b] = gone ? len - gone * p.page : raw;
        }
    }
    const int *ti = p.table + at;
    int *to = a.table_out + at;
    const float *wi = a.weight + at;
    float *wo = a.weight_out + at;
    if (gone == 0) {
        if (row < 0 ? to != ti : wo != wi)
            for (int j = tid; j < P; j += kMoveThreads) {
                if (row < 0)
                    to[j] = ti[j];
                else
                    wo[j] = wi[j];
            }
        return;
    }
    // among the competing pages [first, n - last) the (keep - first - last)-th largest key, and how many of its equals stay
    const uint32_t *keys = a.keys + (long long)b * P;
    const int c0 = a.first, c1 = n - a.last;
    int left = a.keep - a.first - a.last;
    uint32_t last_key = 0xffffffffu;
    if (left > 0) {
        uint32_t found = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kMoveThreads) s_hist[i] = 0;
            __syncthreads();
            for (int j = c0 + tid; j < c1; j += kMoveThreads) {
                const uint32_t k = keys[j];
                if (shift == 24 || (k >> (shift + 8)) == (found >> (shift + 8))) atomicAdd(&s_hist[(k >> shift) & 255], 1);
            }
            __syncthreads();
            if (wid == 0) {  // bins from the top: lane l has bins 255 - 8 l .. 248 - 8 l
                int mine = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) mine += s_hist[255 - 8 * lane - e];
                int inc = mine;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, inc, off);
                    if (lane >= off) inc += y;
                }
                if (inc - mine < left && left <= inc) {  // one lane
                    int before = inc - mine, e = 0;
                    while (before + s_hist[255 - 8 * lane - e] < left) before += s_hist[255 - 8 * lane - e++];
                    s_bin = 255 - 8 * lane - e;
                    s_left = left - before;
                }
            }
            __syncthreads();
            found |= (uint32_t)s_bin << shift;
            left = s_left;
        }
        last_key = found;
    }
    // a page stays that competes with a larger key, that is kept or lies behind the end, or that is among the first
    // `left` of last_key
    int above = 0, equal = 0;  // before this chunk
    for (int j0 = 0; j0 < P; j0 += kMoveThreads) {
        const int j = j0 + tid;
        const bool in = j < P, competes = in && j >= c0 && j < c1;
        const uint32_t k = competes ? keys[j] : 0;
        const bool gt = in && (!competes || k > last_key), eq = competes && left > 0 && k == last_key;
        const int t = in && row < 0 ? ti[j] : 0;
        const float w = in && row >= 0 ? wi[j] : 0.f;
        int inc = (gt ? 1 : 0) | (eq ? 1 << 16 : 0);
        const int mine = inc;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += y;
        }
        if (lane == 31) s_warp[wid] = inc;
        __syncthreads();  // the chunk was read
        int all = 0;
#pragma unroll
        for (int v = 0; v < kMoveWarps; ++v) {
            if (v == wid) inc += all;
            all += s_warp[v];
        }
        const int eq_before = equal + ((inc - mine) >> 16), place = above + ((inc - mine) & 0xffff) + min(eq_before, left);
        if (in && (gt || (eq && eq_before < left))) {
            if (row < 0)
                to[place] = t;
            else
                wo[place] = w;
        } else if (in && row < 0) {
            a.freed[(long long)b * a.freed_cap + (j - place)] = t;
        }
        above += all & 0xffff;
        equal += all >> 16;
        __syncthreads();  // s_warp was read
    }
    for (int j = P - gone + tid; j < P; j += kMoveThreads) {
        if (row < 0)
            to[j] = -1;
        else
            wo[j] = 0.f;
    }
}

}  // namespace
}  // namespace vsa

using namespace vsa;

extern "C" vsa_status vsa_paged_attn_weigh(const vsa_paged_desc *desc, const void *q, int64_t q_stride, const void *k_cache,
                                           const void *v_cache, const float *k_scale, const float *v_scale,
                                           const int32_t *page_idx, const int32_t *page_cnt, int idx_cap, void *out,
                                           float *lse, const float *page_weight, float *weight_out, float decay,
                                           void *workspace, size_t workspace_bytes, vsa_stream_t stream) {
    WeighArgs a{};
    const vsa_status st = to_paged(desc, &a.p, true);
    if (st != VSA_OK) return st;
    if (!page_weight || !weight_out || !k_scale != !v_scale) return VSA_ERR_NULL;
    if (((uintptr_t)page_weight | (uintptr_t)weight_out) & 3u) return VSA_ERR_LAYOUT;
    if (!(decay >= 0.f && decay <= 1.f)) return VSA_ERR_SHAPE;
    if (page_idx && idx_cap > a.p.max_pages) return VSA_ERR_UNSUPPORTED;  // records are kept per page of the table
    const bool eight = k_scale != nullptr;
    const long long chunks = (a.p.max_pages + kWeighThreads - 1) / kWeighThreads;
    const long long ctas = (long long)a.p.B * a.p.Hkv * (page_idx ? 1 : chunks);
    if (ctas > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const AttnCall c{desc, q, q_stride, k_cache, v_cache, k_scale, v_scale, page_idx, page_cnt, idx_cap, out, lse,
                     workspace, workspace_bytes, true};
    const vsa_status done = eight ? attn8(c, s) : attn16(c, s);
    if (done != VSA_OK) return done;
    a.idx = page_idx;
    a.cnt = page_cnt;
    a.cap = idx_cap;
    a.lse = lse;
    a.bw = reinterpret_cast<const float2 *>(static_cast<char *>(workspace) + paged_ws(a.p).total);
    a.blocks = a.p.max_len / 16;
    a.rows = rows_of(a.p.G);
    a.rc = (a.p.G + a.rows - 1) / a.rows;
    a.in = page_weight;
    a.out = weight_out;
    a.decay = decay;
    a.drop = attn_drop(eight, a.p.dtype);
    prof_begin("page_weigh", s);
    const cudaError_t e = launch_paged(page_idx ? k_page_weigh_listed : k_page_weigh, dim3((unsigned)ctas), kWeighThreads, 0, 1,
                                       a, s);
    prof_end(s);
    return status_from_cuda(e);
}

extern "C" vsa_status vsa_page_evict(const vsa_paged_desc *desc, const float *page_weight, int keep, int keep_first,
                                     int keep_last, int32_t *table_out, int32_t *lens_out, float *weight_out, int32_t *freed,
                                     int32_t *freed_cnt, void *workspace, size_t workspace_bytes, vsa_stream_t stream) {
    EvictArgs a{};
    const vsa_status st = to_paged(desc, &a.p, true);
    if (st != VSA_OK) return st;
    if (!page_weight || !table_out || !lens_out || !weight_out || !freed || !freed_cnt) return VSA_ERR_NULL;
    if (((uintptr_t)page_weight | (uintptr_t)table_out | (uintptr_t)lens_out | (uintptr_t)weight_out | (uintptr_t)freed |
         (uintptr_t)freed_cnt) & 3u)
        return VSA_ERR_LAYOUT;
    if (keep_first < 0 || keep_last < 1 || keep < (long long)keep_first + keep_last) return VSA_ERR_SHAPE;
    const PagedWs ws = paged_ws(a.p);
    if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < ws.total) return VSA_ERR_WORKSPACE;
    const long long sums = (long long)a.p.B * ((a.p.max_pages + kSumThreads - 1) / kSumThreads);
    const long long moves = (long long)a.p.B * (a.p.Hkv + 1);
    if (sums > 0x7fffffffLL || moves > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    a.weight = page_weight;
    a.keep = keep;
    a.first = keep_first;
    a.last = keep_last;
    a.freed_cap = keep < a.p.max_pages ? a.p.max_pages - keep : 1;
    a.table_out = table_out;
    a.lens_out = lens_out;
    a.weight_out = weight_out;
    a.freed = freed;
    a.cnt = freed_cnt;
    char *w = static_cast<char *>(workspace);
    a.keys = reinterpret_cast<uint32_t *>(w + ws.keys);
    a.len = reinterpret_cast<int *>(w + ws.seg);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    prof_begin("evict_sums", s);
    cudaError_t e = launch_paged(k_evict_sums, dim3((unsigned)sums), kSumThreads, 0, 1, a, s);
    prof_end(s);
    if (e != cudaSuccess) return status_from_cuda(e);
    prof_begin("evict_move", s);
    e = launch_paged(k_evict_move, dim3((unsigned)moves), kMoveThreads, 0, 1, a, s);
    prof_end(s);
    return status_from_cuda(e);
}
