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
// and values. k_page_weigh puts them over the rows' sums, per page, by the
// difference of the maxima before its scaling: a row's weights are one together
// at any score.
#include <algorithm>

#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace vsa {
namespace {

struct WeighArgs {
    Paged p;
    const int *idx, *cnt;
    int cap;
    const float2 *stat;    // [B, Hq] the rows' maxima of q.k, and 1 / their sums of P
    const float2 *bw;      // [segments, blocks, rows]
    int blocks, rows, rc;
    const float *in;       // [B, Hkv, max_pages]
    float *out;
    float decay, drop;     // drop: the attention's lift of P, undone
    float sl2;             // P's exponent per unit of q.k, in log2 units
    int lanes, row_lanes;  // log2 of the lanes per page (as many as it has records, up to 32), and of those per block
    unsigned chunks;       // CTAs per list row
};
constexpr int kWeighThreads = 256;
constexpr int kWeighDeep = 4;  // pages per group of lanes

// Sum of P over `n` blocks from entry block `blk` of key/value head h of sequence b (list row bh), all of its query heads: by
// the 2^lanes lanes of a group, `me` a lane's place in it. The records of a page lie side by side: a group reads them
// together, a lane those of one row (of `row_lanes` bits; a chunk with fewer rows leaves lanes idle).
__device__ __forceinline__ float mass_of(const WeighArgs &a, int b, int h, int bh, int blk, int n, int me) {
    const Paged &p = a.p;
    const int i = me & ((1 << a.row_lanes) - 1);
    float mass = 0.f;
    for (int r = 0; r < a.rc; ++r) {
        if (i >= min(a.rows, p.G - r * a.rows)) break;
        const float2 row = a.stat[(long long)b * p.Hq + h * p.G + r * a.rows + i];
        const float2 *w = a.bw + (((long long)bh * a.rc + r) * a.blocks + blk) * a.rows + i;
        for (int k = me >> a.row_lanes; k < n; k += 1 << (a.lanes - a.row_lanes)) {
            const float2 x = w[k * a.rows];
            if (x.x != 0.f) mass += x.x * (ptx::ex2((x.y - row.x) * a.sl2) * row.y);
        }
    }
    return mass;
}
// ... over the group, in every lane of it; whole warp.
__device__ __forceinline__ float group_sum(const WeighArgs &a, float x) {
    for (int off = 1; off < 1 << a.lanes; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x * a.drop;
}

// All pages: kWeighDeep pages per group of lanes, whose sums go through shared memory so that weights are read and written
// side by side. 64 sequences of up to 16,000 keys x 8 heads with 4 queries each (94,000 blocks, 512 rows of 250 pages) add
// 5 us to the attention's 74; a thread per page, which reads its records one after another, 14; a weight read and
// written by each group 8.
__global__ void __launch_bounds__(kWeighThreads) k_page_weigh(WeighArgs a) {
    __shared__ float s_sum[kWeighThreads * kWeighDeep];
    const Paged &p = a.p;
    const int per = kWeighThreads >> a.lanes, span = per * kWeighDeep, tid = threadIdx.x;
    const unsigned bh = blockIdx.x / a.chunks, b = bh / (unsigned)p.Hkv, h = bh - b * p.Hkv;
    const int me = tid & ((1 << a.lanes) - 1), slot = tid >> a.lanes, j0 = (int)(blockIdx.x - bh * a.chunks) * span;
    const long long at = (long long)bh * p.max_pages + j0;
    grid_wait();
    grid_go();
    const int len = paged_len(p, (int)b), mine = min(span, p.max_pages - j0);
    if ((long long)j0 << p.page_log2 >= len) {  // behind the sequence's end
        if (a.out != a.in)
            for (int i = tid; i < mine; i += kWeighThreads) a.out[at + i] = a.in[at + i];
        return;
    }
    const float old = tid < mine ? a.in[at + tid] : 0.f;
    float mass[kWeighDeep];
#pragma unroll
    for (int d = 0; d < kWeighDeep; ++d) {
        const int j = j0 + slot + d * per;
        const bool live = j < p.max_pages && j << p.page_log2 < len;
        const int from = live ? j << p.page_log2 : 0;
        mass[d] = live ? mass_of(a, (int)b, (int)h, (int)bh, from >> 4, (min(len - from, p.page) + 15) >> 4, me) : 0.f;
    }
#pragma unroll
    for (int d = 0; d < kWeighDeep; ++d) {
        const float sum = group_sum(a, mass[d]);
        if (me == 0) s_sum[slot + d * per] = sum;
    }
    __syncthreads();
    for (int i = tid; i < mine; i += kWeighThreads) {
        const float was = i == tid ? old : a.in[at + i];
        const bool live = (j0 + i) << p.page_log2 < len;
        a.out[at + i] = !live ? was : a.decay == 0.f ? s_sum[i] : fmaf(a.decay, was, s_sum[i]);
    }
}

// Listed pages: one CTA per list, a few entries per turn. A list that is not ascending may name a page
// twice: its entries are then added one after another. On top of the attention's
// time (us, ascending / any order): 64 sequences x 8 heads, 64 of 250 pages of 64
// tokens, 10 / 26 on 104; 8 x 8 heads with 16 queries each, 500 of 1,000 of 16 tokens,
// 37 / 116 on 37; one sequence, 4,000 of 8,000 of 16 tokens, 1 head 55 / 585 on 12, 8 heads
// 72 / 668 on 32. Chains of loads bound it, in any order one thread's additions; a list
// in parts is not built.
__global__ void __launch_bounds__(kWeighThreads) k_page_weigh_listed(WeighArgs a) {
    __shared__ float s_mass[kWeighThreads];
    const Paged &p = a.p;
    const long long bh = blockIdx.x;
    const int tid = threadIdx.x;
    grid_wait();
    grid_go();
    const int b = (int)(bh / p.Hkv), h = (int)(bh % p.Hkv), len = paged_len(p, b), cnt = clampi(a.cnt[bh], 0, a.cap);
    const int *idx = a.idx + bh * a.cap;
    float *out = a.out + bh * p.max_pages;
    for (int j = tid; j < p.max_pages; j += kWeighThreads) {
        const long long at = bh * p.max_pages + j;
        if ((long long)j << p.page_log2 < len) {
            if (a.decay != 1.f || a.out != a.in) a.out[at] = a.decay == 0.f ? 0.f : a.decay * a.in[at];
        } else if (a.out != a.in) {
            a.out[at] = a.in[at];
        }
    }
    bool ascending = true;
    for (int n = tid + 1; n < cnt; n += kWeighThreads) ascending = ascending && idx[n - 1] < idx[n];
    ascending = __syncthreads_and(ascending);
    const int blocks = p.page / 16, per = kWeighThreads >> a.lanes, me = tid & ((1 << a.lanes) - 1), slot = tid >> a.lanes;
    for (int n0 = 0; n0 < cnt; n0 += per) {
        const int n = n0 + slot, j = n < cnt ? idx[n] : -1;
        const bool on = j >= 0 && j < p.max_pages && (long long)j << p.page_log2 < len;
        const float mass = group_sum(a, on ? mass_of(a, b, h, (int)bh, n * blocks, blocks, me) : 0.f);
        if (ascending) {
            if (on && me == 0) out[j] += mass;
        } else {
            if (me == 0) s_mass[slot] = mass;
            __syncthreads();
            if (tid == 0)
                for (int i = 0; i < per && n0 + i < cnt; ++i) {
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
constexpr int kSumThreads = 256;
// Whether one CTA takes a whole sequence (of up to 1,024 pages) in one launch,
// which costs it half a microsecond or more per head, instead of a launch for the
// sums and then a CTA per row, which does where there are many more rows than SMs.
// Measured (us, one launch / two), 250 pages: 1 sequence x 4, 8, 16, 32 heads 5.8 / 6.1,
// 6.9 / 6.3, 10.5 / 7.9, 18.7 / 10.3; 16 x 8, 32 7.1 / 7.9, 19.6 / 20.0; 24 x 8, 16, 32 7.0 / 9.9,
// 12.0 / 14.6, 19.7 / 26.5; 64 x 1, 8, 32 5.6 / 6.6, 7.7 / 17.9, 19.6 / 66.2. 1,000 pages: 1 x
// 1, 8, 32 9.9 / 5.7, 11.4 / 6.7, 35.4 / 10.6; 24 x 8, 16, 32 12.4 / 11.6, 19.8 / 17.5, 36.1 / 32.7;
// 64 x 1, 4, 32 10.5 / 7.5, 11.3 / 14.6, 36.2 / 79.3.
inline bool one_launch(const Paged &p) {
    if (p.max_pages > 1024) return false;
    return (p.Hkv <= 4 && p.max_pages <= 512) || (p.B > 20 && (long long)p.B * (p.Hkv + 1) > 152);
}

// A float's order as an unsigned's; NaN with -inf, -0 with 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A page's weight over the heads, as a key: added in fp64 in ascending order (k_evict_move adds in the same one where it does
// so itself), rounded once to fp32.
__device__ __forceinline__ uint32_t page_key(const EvictArgs &a, int b, int j) {
    const Paged &p = a.p;
    const float *w = a.weight + (long long)b * p.Hkv * p.max_pages + j;
    double sum = 0.0;
#pragma unroll 8
    for (int h = 0; h < p.Hkv; ++h) sum += (double)w[(long long)h * p.max_pages];
    return order_key((float)sum);
}
__global__ void __launch_bounds__(kSumThreads) k_evict_sums(EvictArgs a) {
    const Paged &p = a.p;
    const int chunks = (p.max_pages + kSumThreads - 1) / kSumThreads;
    const int b = (int)(blockIdx.x / chunks), j = (int)(blockIdx.x % chunks) * kSumThreads + threadIdx.x;
    grid_wait();
    grid_go();
    const int raw = p.lens[b], len = clampi(raw, 0, p.max_len);
    if (j == 0) a.len[b] = raw;
    if (j >= p.max_pages || (long long)j << p.page_log2 >= len) return;
    a.keys[(long long)b * p.max_pages + j] = page_key(a, b, j);
}

// Places the pages of sequence b and moves rows of it (row -1: the table, 0 .. Hkv - 1: a head's weights), N threads with E
// entries each, N apart. One: the CTA has all rows and makes the keys itself, each thread one page; otherwise it has
// one row, with the keys made before.
//
// The last key to stay: 11 bits at a time from the top (2,048 bins: weights share their exponents, and one bin of few
// takes the additions of a warp one after another), until a bin stays as a whole or its keys are all equal. Then the
// counts of all warps, N E entries at a time, place them. An entry moves to a place at or before its own, and a chunk is read before any of it is
// written, so a row may be moved in place. What will be moved is loaded first of all.
//
// Chains of loads and barriers bound it: 64 sequences of up to 250 pages x 8 heads 6.9 us in one launch (7.9 with the keys
// before each counted instead of the digits); one of 7,680 pages x 24 heads 13.2, 4 of them the sums. With 8-bit digits and
// 512 entries placed at a time the latter took 18.9, 25 where a warp's lanes matched their bins first, and 15.9 with a
// thread's entries side by side, whose stores are not.
// Rows of a sequence loaded at once: 8, 10, 16 took 6.0, 6.9, 7.3 us for 64 sequences of 250 pages x 4 heads, 7.9, 7.0, 8.2
// for 8 heads (nine rows: all at once with ten), 12.0, 12.1, 11.2 for 16, 19.5, 19.8, 19.2 for 32.
constexpr int kBins = 2048, kRowsAhead = 10;
template <int N, int E, bool kOne> __global__ void __launch_bounds__(N) k_evict_move(EvictArgs a) {
    constexpr int W = N / 32, kChunk = N * E, R = kOne ? kRowsAhead : 1;
    static_assert(!kOne || E == 1, "one page per thread");
    __shared__ int s_hist[kBins];
    __shared__ int s_bin, s_left, s_in, s_warp[W], s_cnt[E * W], s_all;
    const Paged &p = a.p;
    const int rows = kOne ? 1 : p.Hkv + 1;  // CTAs per sequence
    const int b = (int)(blockIdx.x / rows), row0 = (int)(blockIdx.x - (unsigned)b * rows) - 1;
    const int row1 = kOne ? p.Hkv : row0 + 1;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, P = p.max_pages;
    auto from = [&](int row) -> const int * {
        return row < 0 ? p.table + (long long)b * P
                       : reinterpret_cast<const int *>(a.weight) + ((long long)b * p.Hkv + row) * P;
    };
    auto to = [&](int row) -> int * {
        return row < 0 ? a.table_out + (long long)b * P
                       : reinterpret_cast<int *>(a.weight_out) + ((long long)b * p.Hkv + row) * P;
    };
    grid_wait();
    grid_go();
    int x[R][E];  // the first chunk of the first rows
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < E; ++e) x[r][e] = row0 + r < row1 && e * N + tid < P ? from(row0 + r)[e * N + tid] : 0;
    const int raw = kOne ? p.lens[b] : a.len[b], len = clampi(raw, 0, p.max_len), n = (len + p.page - 1) >> p.page_log2;
    const int gone = n > a.keep ? n - a.keep : 0;
    const int c0 = a.first, c1 = n - a.last;  // the pages that compete
    auto key_at = [&](int j) { return a.keys[(long long)b * P + j]; };
    uint32_t key[E];
    if constexpr (kOne) {
        double sum = 0.0;  // page_key's order
#pragma unroll
        for (int r = 1; r < R; ++r) sum += row0 + r < row1 ? (double)__int_as_float(x[r][0]) : 0.0;
#pragma unroll 8
        for (int row = row0 + R; row < row1; ++row) sum += tid < P ? (double)__int_as_float(from(row)[tid]) : 0.0;
        key[0] = order_key((float)sum);
    } else if (gone) {
#pragma unroll
        for (int e = 0; e < E; ++e) key[e] = e * N + tid >= c0 && e * N + tid < c1 ? key_at(e * N + tid) : 0;
    }
    if (row0 < 0) {
        for (int i = gone + tid; i < a.freed_cap; i += N) a.freed[(long long)b * a.freed_cap + i] = -1;
        if (tid == 0) a.cnt[b] = gone;
    }
    if (gone == 0) {
        if (row0 < 0 && tid == 0) a.lens_out[b] = raw;
        for (int row = row0; row < row1; ++row)
            if (to(row) != from(row))
                for (int j = tid; j < P; j += N) to(row)[j] = from(row)[j];
        return;
    }
    // a page that competes stays with a key above `last_key`, or as one of the first `left` equal to it
    int left = a.keep - a.first - a.last;
    uint32_t last_key = 0xffffffffu;
    if (left > 0) {
        uint32_t found = 0;
        int shift = 21, known = 32;  // the digit's place; `known`: bits below it and its own
        for (;;) {
            const int bits = known - shift, bins = 1 << bits;
            for (int i = tid; i < kBins; i += N) s_hist[i] = 0;
            __syncthreads();
            auto count = [&](int j, uint32_t k) {
                if (j >= c0 && j < c1 && (known == 32 || k >> known == found >> known))
                    atomicAdd(&s_hist[k >> shift & (bins - 1)], 1);
            };
#pragma unroll
            for (int e = 0; e < E; ++e) count(e * N + tid, key[e]);
            if constexpr (!kOne)
                for (int j = kChunk + tid; j < c1; j += N) count(j, j >= c0 ? key_at(j) : 0);
            __syncthreads();
            // bins from the top, kBins / N or so to a thread: their sums before it, and the thread that holds the last one
            constexpr int kPer = kBins / N > 0 ? kBins / N : 1;
            int mine = 0;
            if (tid * kPer < kBins)
#pragma unroll
                for (int e = 0; e < kPer; ++e) mine += s_hist[kBins - 1 - tid * kPer - e];
            int inc = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += y;
            }
            if (lane == 31) s_warp[wid] = inc;
            __syncthreads();
            inc += __reduce_add_sync(0xffffffffu, lane < wid ? s_warp[lane] : 0);
            if (inc - mine < left && left <= inc) {  // one thread
                int before = inc - mine, at = kBins - 1 - tid * kPer;
                while (before + s_hist[at] < left) before += s_hist[at--];
                s_bin = at;
                s_left = left - before;
                s_in = s_hist[at];
            }
            __syncthreads();
            found |= (uint32_t)s_bin << shift;
            left = s_left;
            if (s_in == left && found) {  // the bin stays as a whole
                last_key = found - 1;
                left = 0;
                break;
            }
            if (shift == 0) {
                last_key = found;
                break;
            }
            known = shift;
            shift = shift > 11 ? shift - 11 : 0;
        }
    }
    int above = 0, equal = 0;  // before this chunk
    for (int j0 = 0; j0 < P; j0 += kChunk) {
        int place[E];  // ~ its number among the freed ones where it goes
        unsigned gt[E], eq[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = j0 + e * N + tid;
            const bool competes = j >= c0 && j < c1;
            const uint32_t k = !competes ? 0 : j0 == 0 ? key[e] : kOne ? 0 : key_at(j);
            gt[e] = __ballot_sync(0xffffffffu, j < P && (!competes || k > last_key));
            eq[e] = __ballot_sync(0xffffffffu, competes && left > 0 && k == last_key);
            if (lane == 0) s_cnt[e * W + wid] = __popc(gt[e]) | __popc(eq[e]) << 16;  // in the order of j; kChunk < 2^15
        }
        __syncthreads();
        if (wid == 0) {  // the counts before each
            constexpr int kPer = (E * W + 31) / 32;
            int mine[kPer], sum = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                mine[i] = lane * kPer + i < E * W ? s_cnt[lane * kPer + i] : 0;
                sum += mine[i];
            }
            int inc = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += y;
            }
            if (lane == 31) s_all = inc;
            inc -= sum;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (lane * kPer + i < E * W) s_cnt[lane * kPer + i] = inc;
                inc += mine[i];
            }
        }
        __syncthreads();
        const unsigned before = (1u << lane) - 1;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = j0 + e * N + tid, cnt = s_cnt[e * W + wid];
            const int g = above + (cnt & 0xffff) + __popc(gt[e] & before), q = equal + (cnt >> 16) + __popc(eq[e] & before);
            const int at = g + min(q, left);
            place[e] = (gt[e] >> lane & 1) || ((eq[e] >> lane & 1) && q < left) ? at : ~(j - at);
        }
        above += s_all & 0xffff;
        equal += s_all >> 16;
        for (int row = row0; row < row1; row += R) {
            if (j0 > 0 || row > row0) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        x[r][e] = row + r < row1 && j0 + e * N + tid < P ? from(row + r)[j0 + e * N + tid] : 0;
            }
            __syncthreads();  // the chunk of these rows was read (and the counts)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (row + r >= row1 || j0 + e * N + tid >= P) continue;
                    if (place[e] >= 0)
                        to(row + r)[place[e]] = x[r][e];
                    else if (row + r < 0)
                        a.freed[(long long)b * a.freed_cap + ~place[e]] = x[r][e];
                }
        }
    }
    __syncthreads();
    if (row0 < 0 && tid == 0) a.lens_out[b] = len - gone * p.page;  // which may be where every thread read raw
    for (int row = row0; row < row1; ++row)
        for (int j = P - gone + tid; j < P; j += N) to(row)[j] = row < 0 ? -1 : 0;  // 0.f
}

template <int N, int E, bool kOne> cudaError_t launch_evict(const EvictArgs &a, cudaStream_t s) {
    prof_begin("evict_move", s);
    const cudaError_t e = launch_paged(k_evict_move<N, E, kOne>, dim3((unsigned)(kOne ? a.p.B : a.p.B * (a.p.Hkv + 1))), N, 0, 1,
                                       a, s);
    prof_end(s);
    return e;
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
    a.rows = rows_of(a.p.G);
    while (1 << a.row_lanes < a.rows) ++a.row_lanes;
    a.lanes = std::min(a.row_lanes + a.p.page_log2 - 4, 5);
    const int span = (kWeighThreads >> a.lanes) * kWeighDeep;
    const long long chunks = a.chunks = (unsigned)((a.p.max_pages + span - 1) / span);
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
    const PagedWs ws = paged_ws(a.p);
    a.stat = reinterpret_cast<const float2 *>(static_cast<char *>(workspace) + ws.stat);
    a.bw = reinterpret_cast<const float2 *>(static_cast<char *>(workspace) + ws.total);
    a.sl2 = a.p.scale * kLog2e;
    a.blocks = a.p.max_len / 16;
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
    const int P = a.p.max_pages;
    if (one_launch(a.p))
        return status_from_cuda(P <= 256 ? launch_evict<256, 1, true>(a, s)
                                : P <= 512 ? launch_evict<512, 1, true>(a, s) : launch_evict<1024, 1, true>(a, s));
    prof_begin("evict_sums", s);
    const cudaError_t e = launch_paged(k_evict_sums, dim3((unsigned)sums), kSumThreads, 0, 1, a, s);
    prof_end(s);
    if (e != cudaSuccess) return status_from_cuda(e);
    return status_from_cuda(P <= 1024 ? launch_evict<1024, 1, false>(a, s)
                            : P <= 4096 ? launch_evict<1024, 4, false>(a, s) : launch_evict<1024, 8, false>(a, s));
}
