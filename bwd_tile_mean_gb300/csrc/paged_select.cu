// paged_select.cu -- the pages each key/value head attends to, by the score
// of their mean key against the group's query (vsa_page_select).
//
// A page competes unless it is among the first keep_first or the last
// keep_last. Its fp32 mean is read once (8 lanes per page, 16 bytes per load,
// through a ring of asynchronous copies per warp; the heads of a page are
// neighbours in memory; a lane reads back what it copied itself) and becomes
// one order-preserving 32-bit key per head. Then a CTA per row finds the last
// page to take under (key desc, page asc), 11 bits of (key, page) at a time
// from the top (a 2,048-bin histogram), until the bin that holds it is small
// enough to rank outright, and lists the taken pages in order.
//
// Few pages, or very many (by_clusters): k_page_select, one launch. A cluster of
// 8 CTAs has one sequence and up to 8 heads, cuts the pages into 8 runs and stores
// the keys straight into the shared memory of the CTA that finishes the head;
// the scores never leave the SMs.
// Others: k_page_scores deals the pages of the whole batch, four at a time with
// up to 16 heads of each, to the CTAs in equal contiguous runs whatever the
// lengths, with the keys in the workspace, and k_page_topk finishes the rows.
// The longest sequence then does not wait for the 8 CTAs of its cluster.
//
// Measured (us, cluster / runs): 960 pages x 24 heads of one sequence 7.7 /
// 11.3, 32 sequences of 312 to 2,047 pages x 8 heads 44 / 30.5. The latter
// reads 105 MB, 15.5 us at the measured copy rate: the means stream in about
// 16 us, before them 4 us go by from the launch (scan of the lengths, page
// ids) and after them 7 to 8 (keys out, the second launch, the top-k). One
// sequence is a chain of loads and barriers: 1.2 us length and page ids, 2.4
// the means, 3 the top-k.
#include <algorithm>

#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace vsa {
namespace {

struct SelectArgs {
    Paged p;
    const void *q;
    long long qs;
    const float *mean;
    int topk, first, last;
    int *idx, *cnt;
    uint32_t *keys;   // [B * Hkv, max_pages] of the competing pages, from keep_first on
    int hg, hgroups;  // heads taken together, and their groups per sequence
    int cap;          // pages per CTA at most
};

constexpr int kThreads = 256, kWarpsSel = kThreads / 32;
constexpr int kTopkThreads = 512;  // 256, 512, 1,024 measured 36.4, 34.9, 34.9 us on 32 sequences of up to 2,047 pages
constexpr int kLongRow = 20480;    // pages from which a row has twice the threads: 512, 1,024 measured 13.5, 14.7 us on one
                                   // of 10,000 pages, 20.0, 20.1 of 20,000, 41.9, 35.0 of 40,000
constexpr int kCtasSel = 304;  // two per SM on 152 SMs
constexpr int kHeads = 16;     // heads of a page taken together at most, in equal groups
constexpr int kLeadSel = 6;    // units a sequence counts for beyond its own (its start-up time): 1, 2, 4, 6 measured
                               // 36.4, 35.6, 34.9, 34.1 us on the same
constexpr int kRing = 5;       // ring stages per warp, each four pages' means of one head (2 KB)
constexpr int kRingBytes = kRing * 2048;
constexpr int kSmemSel = kWarpsSel * kRingBytes + kHeads * kD * 4;
constexpr int kCluster = 8;
constexpr int kClusterStages = 4, kClusterRing = kClusterStages * 2048;
constexpr int kClusterPages = 2048, kFullClusterPages = 2700;  // pages x heads a cluster has at most, the latter where
                                                               // its CTAs fill the GPU
constexpr long long kBatchPages = 560000;  // pages x heads of a batch (290 MB)
constexpr int kBins = 2048;
constexpr int kRank = 256;     // a bin of up to this many pages is ranked outright
constexpr int kIndexBits = 27; // of a page index

// Competing pages of sequence b (all of them full: the partial page is the
// last); 0 when every page is taken.
__device__ __forceinline__ int competing(const SelectArgs &a, int b) {
    const int pages = (paged_len(a.p, b) + a.p.page - 1) >> a.p.page_log2;
    return pages > a.topk ? pages - a.first - a.last : 0;
}

// Larger score, larger key; -0 folded into +0, NaN counted as -inf.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) x = -INFINITY;
    if (x == 0.f) x = 0.f;
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Sums of the group's 16-bit queries at eight dims: fp32 running sums with
// their rounding errors kept aside (each found exactly), added at the end.
template <typename T> __device__ __forceinline__ void group_sum(const T *q, int G, float *out) {
    float s[8], err[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = err[e] = 0.f;
    constexpr int kDeep = 8;  // rows' loads at a time
    for (int m0 = 0; m0 < G; m0 += kDeep) {
        uint4 w[kDeep];
#pragma unroll
        for (int m = 0; m < kDeep; ++m)
            w[m] = m0 + m < G ? *reinterpret_cast<const uint4 *>(q + (long long)(m0 + m) * kD) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int m = 0; m < kDeep; ++m) {
            if (m0 + m >= G) break;
            const uint32_t r[4] = {w[m].x, w[m].y, w[m].z, w[m].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 f = unpack2<T>(r[e / 2]);
                const float x = e & 1 ? f.y : f.x;
                const float t = __fadd_rn(s[e], x), y = __fsub_rn(t, s[e]);
                err[e] = __fadd_rn(err[e], __fadd_rn(__fsub_rn(s[e], __fsub_rn(t, y)), __fsub_rn(x, y)));
                s[e] = t;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = isfinite(s[e]) ? __fadd_rn(s[e], err[e]) : s[e];
}

// (key, page) as one number, the larger the better: 32 key bits, then the
// page counted from the end.
__device__ __forceinline__ uint64_t rank_of(uint32_t key, int c) {
    return ((uint64_t)key << kIndexBits) | (uint32_t)((1 << kIndexBits) - 1 - c);
}

// Score of a page: lane j of eight holds dims 32 i + 4 j + c of its mean, at
// m + 512 i bytes; g: the head's summed query. Every lane gets the score.
__device__ __forceinline__ float page_score(const float *g, const unsigned char *m, int j) {
    float x[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 u = *reinterpret_cast<const float4 *>(g + 32 * i + 4 * j);
        const float4 v = *reinterpret_cast<const float4 *>(m + i * 512);
        x[i][0] = __fmul_rn(u.x, v.x);
        x[i][1] = __fmul_rn(u.y, v.y);
        x[i][2] = __fmul_rn(u.z, v.z);
        x[i][3] = __fmul_rn(u.w, v.w);
    }
    // 128 -> 64 -> 32: dims 64 and 32 apart; then neighbours
    float y[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) y[d] = __fadd_rn(__fadd_rn(x[0][d], x[2][d]), __fadd_rn(x[1][d], x[3][d]));
    float r = __fadd_rn(__fadd_rn(y[0], y[1]), __fadd_rn(y[2], y[3]));
    r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 1));
    r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 2));
    return __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 4));
}
// Four pages' means of one head into a ring stage; page: this lane's, -1: zeros.
__device__ __forceinline__ void copy_means(uint32_t dst, const SelectArgs &a, int page, int head, int j) {
    const float *src = a.mean + ((long long)max(page, 0) * a.p.Hkv + head) * kD + 4 * j;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * 512), "l"(src + 32 * i),
                     "r"(page >= 0 ? 16 : 0)
                     : "memory");
}

// A warp's items: four pages of one of hn heads each, every kWarpsSel-th item
// from its own number on, without a division per item.
struct Walk {
    int head, quad, dh, dq, hn;
    __device__ __forceinline__ Walk(int first, int heads)
        : head(first % heads), quad(first / heads), dh(kWarpsSel % heads), dq(kWarpsSel / heads), hn(heads) {}
    __device__ __forceinline__ void next() {
        head += dh;
        quad += dq;
        if (head >= hn) {
            head -= hn;
            ++quad;
        }
    }
};

template <typename T> __global__ void __launch_bounds__(kThreads) k_page_scores(SelectArgs a) {
    extern __shared__ __align__(16) unsigned char sm[];
    float *sq = reinterpret_cast<float *>(sm + kWarpsSel * kRingBytes);  // [kHeads][128] summed queries
    const Paged &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    grid_wait();
    // a unit: four pages, the heads of one group; a group's lead goes before its own units
    auto units_of = [&](int n) { const int q = (competing(a, n) + 3) / 4; return q > 0 ? q + kLeadSel : 0; };
    const Run run = find_run<kWarpsSel>(
        p.B, [&](int n) -> long long { return (long long)units_of(n) * a.hgroups; }, kCtasSel, 1, 1);
    long long before = run.before;
    int b = run.n;
    for (long long x = run.x0; x < run.x1 && b < p.B;) {
        const int comp = competing(a, b), units = units_of(b);
        if (x >= before + (long long)units * a.hgroups) {
            before += (long long)units * a.hgroups;
            ++b;
            continue;
        }
        const int grp = div_small(x - before, units), off = (int)(x - before - (long long)grp * units);
        const int take = (int)min((long long)(units - off), run.x1 - x);
        const int q0 = max(off - kLeadSel, 0), nq = max(off + take - kLeadSel, 0) - q0;  // its own units
        const int h0 = grp * a.hg, hn = min(a.hg, p.Hkv - h0);
        x += take;
        if (nq == 0) continue;

        // An item is four pages of one head; lane j of eight holds dims 32 i + 4 j + c of a page.
        const int sub = lane >> 3, j = lane & 7, items = nq * hn;
        const uint32_t ring = ptx::smem_addr(sm) + wid * kRingBytes + lane * 16;
        int id[kRing], at[kRing], head[kRing];  // of the items in flight, by stage: page id, competing page, head
        Walk w(wid, hn);
        auto plan = [&](int stage) {  // the next item
            at[stage] = (q0 + w.quad) * 4 + sub;
            head[stage] = w.head;
            id[stage] = w.quad < nq && at[stage] < comp ? paged_id(p, b, a.first + at[stage]) : -1;
            w.next();
        };
        auto copy = [&](int stage) { copy_means(ring + stage * 2048, a, id[stage], h0 + head[stage], j); };
#pragma unroll
        for (int s = 0; s < kRing; ++s) plan(s);
#pragma unroll
        for (int s = 0; s < kRing - 1; ++s) {
            if (wid + s * kWarpsSel < items) copy(s);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        __syncthreads();  // the sums of the piece before were read
        const T *q = static_cast<const T *>(a.q) + b * a.qs + (long long)h0 * p.G * kD;
        if (tid < hn * (kD / 8)) group_sum<T>(q + (long long)(tid >> 4) * p.G * kD + 8 * (tid & 15), p.G, sq + 8 * tid);
        __syncthreads();
        uint32_t *keys = a.keys + ((long long)b * p.Hkv + h0) * p.max_pages;
        for (int n0 = 0; wid + n0 * kWarpsSel < items; n0 += kRing) {
#pragma unroll
            for (int s = 0; s < kRing; ++s) {
                const int it = wid + (n0 + s) * kWarpsSel;
                if (it >= items) break;
                const int sa = (s + kRing - 1) % kRing;
                if (it + (kRing - 1) * kWarpsSel < items) copy(sa);  // into the stage this lane read last
                asm volatile("cp.async.commit_group;" ::: "memory");
                asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
                const int hh = head[s], c = at[s], page = id[s];
                plan(s);
                const float r = page_score(sq + hh * kD, sm + wid * kRingBytes + s * 2048 + lane * 16, j);
                if (j == 0 && c < comp) keys[(long long)hh * p.max_pages + c] = order_key(page >= 0 ? r : -INFINITY);
            }
        }
    }
    grid_go();
}

// Rows with nothing to choose: every page.
template <int N> __device__ __forceinline__ void list_all(const SelectArgs &a, long long row, int pages) {
    for (int n = threadIdx.x; n < a.topk; n += N) a.idx[row * a.topk + n] = n < pages ? n : -1;
    if (threadIdx.x == 0) a.cnt[row] = pages;
}
template <int N> __device__ __forceinline__ void clear_bins(int (&hist)[kBins]) {
    for (int e = threadIdx.x; e < kBins / 4; e += N) reinterpret_cast<int4 *>(hist)[e] = make_int4(0, 0, 0, 0);
}

// Lists the pages of a row: the first and last ones that are always taken,
// and the `take` best of the competing ones, whose keys are keys[0, comp).
// Whole CTA; `hist` is clear.
template <int N>
__device__ __forceinline__ void list_pages(const SelectArgs &a, long long row, int pages, int comp, int (&hist)[kBins],
                                           const uint32_t *keys) {
    constexpr int W = N / 32;
    __shared__ int wsum[W];
    __shared__ int s_bin, s_above, s_in, s_fill;
    __shared__ uint64_t s_cut;
    __shared__ uint64_t list[kRank];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int take = a.topk - a.first - a.last;
    int *idx = a.idx + row * a.topk;
    // f(rank) of this thread's share of the pages, kDeep loads at a time
    constexpr int kDeep = 8;
    auto each = [&](auto f) {
        for (int c0 = tid; c0 < comp; c0 += N * kDeep) {
            uint32_t key[kDeep];
#pragma unroll
            for (int e = 0; e < kDeep; ++e) key[e] = c0 + e * N < comp ? keys[c0 + e * N] : 0u;
#pragma unroll
            for (int e = 0; e < kDeep; ++e)
                if (c0 + e * N < comp) f(rank_of(key[e], c0 + e * N));
        }
    };
    // cut: the `take`-th largest rank (ranks are distinct); 2^59 when none is taken. Every pass fixes more bits, so
    // the loop ends whatever the keys are.
    uint64_t cut = 1ull << (32 + kIndexBits), prefix = 0;
    int rem = take;
    for (int top = 32 + kIndexBits; rem > 0 && top > 0;) {  // bits [top, 59) of the cut are `prefix`
        const int shift = max(top - 11, 0), bits = top - shift;
        __syncthreads();  // the bins are clear (and the keys there)
        each([&](uint64_t k) {
            if (k >> top == prefix) atomicAdd(&hist[(int)((k >> shift) & ((1u << bits) - 1u))], 1);
        });
        __syncthreads();
        // thread t: the bins 2047 - kPer t and down
        constexpr int kPer = kBins / N;
        int cnt[kPer], sum = 0;
#pragma unroll
        for (int e = 0; e < kPer; e += 2) {
            const int2 n = *reinterpret_cast<const int2 *>(&hist[kBins - 2 - tid * kPer - e]);
            cnt[e] = n.y, cnt[e + 1] = n.x;
            sum += n.x + n.y;
        }
        int inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += y;
        }
        if (lane == 31) wsum[wid] = inc;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) inc += w < wid ? wsum[w] : 0;
        int above = inc - sum;  // pages in larger bins
        if (above < rem && inc >= rem) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (above < rem) {
                    s_bin = kBins - 1 - tid * kPer - e;
                    s_above = above;
                    s_in = cnt[e];
                    above += cnt[e];
                }
        }
        if (tid == 0) s_fill = 0;
        __syncthreads();
        prefix = (prefix << bits) | (uint32_t)s_bin;
        top = shift;
        rem -= s_above;
        const int in = s_in;
        if (in == rem) {  // the whole bin
            cut = prefix << top;
            break;
        }
        if (in <= kRank) {
            each([&](uint64_t k) {
                if (k >> top != prefix) return;
                const int at = atomicAdd(&s_fill, 1);
                if (at < kRank) list[at] = k;
            });
            __syncthreads();
            if (tid < in) {
                const uint64_t k = list[tid];
                int larger = 0;
#pragma unroll 8
                for (int e = 0; e < in; ++e) larger += list[e] > k ? 1 : 0;
                if (larger == rem - 1) s_cut = k;
            }
            __syncthreads();
            cut = s_cut;
            break;
        }
        clear_bins<N>(hist);
    }
    // pages at or above the cut, in order: each warp has a contiguous share
    const int share = ((comp + W - 1) / W + 31) & ~31;
    const int lo = min(wid * share, comp), hi = min(lo + share, comp);
    // chosen(c, ballot) of 32 pages at a time, in order, four loads at a time
    auto each32 = [&](auto f) {
        for (int c0 = lo; c0 < hi; c0 += 128) {
            uint32_t key[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) key[e] = c0 + 32 * e + lane < hi ? keys[c0 + 32 * e + lane] : 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = c0 + 32 * e + lane;
                const bool on = c < hi && rank_of(key[e], c) >= cut;
                f(c, on, __ballot_sync(0xffffffffu, on));
            }
        }
    };
    int n = 0;
    each32([&](int, bool, unsigned m) { n += __popc(m); });
    __syncthreads();  // wsum was read
    if (lane == 0) wsum[wid] = n;
    __syncthreads();
    int at = a.first;
#pragma unroll
    for (int w = 0; w < W; ++w) at += w < wid ? wsum[w] : 0;
    each32([&](int c, bool on, unsigned m) {
        const int to = at + __popc(m & ((1u << lane) - 1u));
        if (on && to < a.topk - a.last) idx[to] = a.first + c;
        at += __popc(m);
    });
    for (int e = tid; e < a.first; e += N) idx[e] = e;
    for (int e = tid; e < a.last; e += N) idx[a.topk - a.last + e] = pages - a.last + e;
    if (tid == 0) a.cnt[row] = a.topk;
}

template <int N> __global__ void __launch_bounds__(N) k_page_topk(SelectArgs a) {
    __shared__ __align__(16) int hist[kBins];
    const Paged &p = a.p;
    const long long row = blockIdx.x;
    const int b = (int)(row / p.Hkv);
    clear_bins<N>(hist);
    grid_wait();
    grid_go();
    const int pages = (paged_len(p, b) + p.page - 1) >> p.page_log2, comp = competing(a, b);
    if (comp == 0)
        list_all<N>(a, row, pages);
    else
        list_pages<N>(a, row, pages, comp, hist, a.keys + row * p.max_pages);
}

template <typename T> __global__ void __launch_bounds__(kThreads) k_page_select(SelectArgs a) {
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ __align__(16) int hist[kBins];
    float *sq = reinterpret_cast<float *>(sm + kWarpsSel * kClusterRing);  // [hg][128] summed queries
    uint32_t *mine = reinterpret_cast<uint32_t *>(sq + a.hg * kD);       // [kCluster * cap] keys of this CTA's head
    int *ids = reinterpret_cast<int *>(mine + kCluster * a.cap);         // [cap] page ids of this CTA's run
    const Paged &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = (int)ptx::cluster_rank(), cl = (int)blockIdx.x / kCluster;
    const int b = cl / a.hgroups, h0 = (cl % a.hgroups) * a.hg, hn = min(a.hg, p.Hkv - h0);
    clear_bins<kThreads>(hist);
    grid_wait();
    const int pages = (paged_len(p, b) + p.page - 1) >> p.page_log2;
    const int comp = competing(a, b);
    if (comp == 0) {
        if (rank < hn) list_all<kThreads>(a, (long long)b * p.Hkv + h0 + rank, pages);
        ptx::cluster_sync();  // with the others, so that a CTA's shared memory is there whatever length they read
        ptx::cluster_sync();
        return;
    }
    const int run = (comp + kCluster - 1) / kCluster;
    const int c0 = min(rank * run, comp), nc = min(run, comp - c0);

    for (int c = tid; c < nc; c += kThreads) ids[c] = paged_id(p, b, a.first + c0 + c);
    const T *q = static_cast<const T *>(a.q) + b * a.qs + (long long)h0 * p.G * kD;
    if (tid < hn * (kD / 8)) group_sum<T>(q + (long long)(tid >> 4) * p.G * kD + 8 * (tid & 15), p.G, sq + 8 * tid);
    ptx::cluster_sync();  // every CTA of the cluster runs: their shared memory may be written

    // An item is four pages of one head; lane j of eight holds dims 32 i + 4 j + c of a page.
    const int sub = lane >> 3, j = lane & 7, items = (nc + 3) / 4 * hn;
    const uint32_t ring = ptx::smem_addr(sm) + wid * kClusterRing + lane * 16;
    Walk w(wid, hn), ahead(wid, hn);  // the item being scored, and the next to copy
    auto copy = [&](int stage) {
        const int c = ahead.quad * 4 + sub;
        copy_means(ring + stage * 2048, a, c < nc ? ids[c] : -1, h0 + ahead.head, j);
        ahead.next();
    };
#pragma unroll
    for (int s = 0; s < kClusterStages - 1; ++s) {
        if (wid + s * kWarpsSel < items) copy(s);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (int n = 0; wid + n * kWarpsSel < items; ++n, w.next()) {
        if (wid + (n + kClusterStages - 1) * kWarpsSel < items)
            copy((n + kClusterStages - 1) % kClusterStages);  // the stage this lane read last
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(kClusterStages - 1) : "memory");
        const int hh = w.head, c = w.quad * 4 + sub;
        const float r = page_score(sq + hh * kD, sm + wid * kClusterRing + (n % kClusterStages) * 2048 + lane * 16, j);
        if (j == 0 && c < nc)
            st_cluster(ptx::cluster_addr(ptx::smem_addr(mine + c0 + c), hh), order_key(ids[c] >= 0 ? r : -INFINITY));
    }
    ptx::cluster_sync();  // every run's keys are there
    grid_go();
    if (rank >= hn) return;

    list_pages<kThreads>(a, (long long)b * p.Hkv + h0 + rank, pages, comp, hist, mine);
}

// CTAs of k_page_select with a.hg heads per cluster.
long long cluster_ctas(const SelectArgs &a) { return (long long)a.p.B * ((a.p.Hkv + a.hg - 1) / a.hg) * kCluster; }

// Whether k_page_select takes the call, and a.hg, a.hgroups for it. Measured
// (us, clusters / equal runs): 960 pages x 24 heads of one sequence 7.7 / 11.3,
// 3 sequences of 580 pages x 40 heads 10.4 / 12.4, 4,984 pages x 3 heads of one
// 11.8 / 10.2, 32 sequences of 312 to 2,047 pages x 8 heads 44 / 30.5. With
// work for many waves of clusters (kBatchPages) those start as others end,
// which evens out the SMs' different shares of the memory (equal runs end
// between 119,000 and 164,000 cycles): 89 sequences of 62 to 1,257 pages x 40
// heads 230 / 282, 20 of 414 to 3,397 x 24 97 / 116, 77 of 162 to 3,025 x 8
// 100.8 / 116.8; with short sequences their own start-up is too much, 89 of 14
// to 195 x 40 82.6 / 68.2.
bool by_clusters(SelectArgs &a) {
    const int pages = a.p.max_pages;
    auto heads = [&](long long ctas, int least) {  // as many per cluster as leave that many CTAs
        for (a.hg = 8; a.hg > least && (cluster_ctas(a) < ctas || a.hg / 2 >= a.p.Hkv);) a.hg /= 2;
        a.hgroups = (a.p.Hkv + a.hg - 1) / a.hg;
        return cluster_ctas(a);
    };
    if (pages >= 400 && pages <= 8192 && (long long)a.p.B * a.p.Hkv * pages > kBatchPages && a.p.Hkv > 1 &&
        heads(700, 2) >= 700)
        return cluster_ctas(a) <= 0x7fffffffLL;
    heads(120, 1);
    auto fits = [&] { return (long long)pages * a.hg <= (cluster_ctas(a) >= 144 ? kFullClusterPages : kClusterPages); };
    while (a.hg > 1 && !fits()) a.hg /= 2;  // fewer heads for each, as far as places last
    a.hgroups = (a.p.Hkv + a.hg - 1) / a.hg;
    return fits() && cluster_ctas(a) <= 320;
}

}  // namespace
}  // namespace vsa

extern "C" vsa_status vsa_page_select(const vsa_paged_desc *desc, const void *q, int64_t q_stride,
                                      const float *k_mean, int topk, int keep_first, int keep_last,
                                      int32_t *page_idx, int32_t *page_cnt, void *workspace, size_t workspace_bytes,
                                      vsa_stream_t stream) {
    using namespace vsa;
    SelectArgs a{};
    const vsa_status st = to_paged(desc, &a.p, true);
    if (st != VSA_OK) return st;
    if (!token_stride(q_stride, a.p.Hq, &a.qs)) return VSA_ERR_SHAPE;
    if (keep_first < 0 || keep_last < 1 || topk < 1 || (long long)keep_first + keep_last > topk) return VSA_ERR_SHAPE;
    // as vsa_paged_attn's lists; the kernels count a list's entries, past its end by a CTA's threads, in 32 bits
    if ((long long)topk * a.p.page > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    if (!q || !k_mean || !page_idx || !page_cnt) return VSA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_mean) || ((uintptr_t)page_idx | (uintptr_t)page_cnt) & 3u) return VSA_ERR_LAYOUT;
    const PagedWs ws = paged_ws(a.p);
    if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < ws.total) return VSA_ERR_WORKSPACE;
    a.q = q;
    a.mean = k_mean;
    a.topk = topk;
    a.first = keep_first;
    a.last = keep_last;
    a.idx = page_idx;
    a.cnt = page_cnt;
    a.keys = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + ws.keys);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool bf = a.p.dtype == T_BF16;
    auto run = [&](const char *name, auto kernel, dim3 grid, int threads, size_t smem, unsigned cluster) {
        cudaError_t e = ensure_smem_limit((const void *)kernel, (int)smem);
        if (e != cudaSuccess) return status_from_cuda(e);
        prof_begin(name, s);
        e = launch_paged(kernel, grid, threads, smem, cluster, a, s);
        prof_end(s);
        return status_from_cuda(e);
    };
    if (a.p.max_pages > topk) {  // otherwise no row has anything to choose
        if (by_clusters(a)) {
            a.cap = (a.p.max_pages + kCluster - 1) / kCluster;
            const size_t smem = kWarpsSel * kClusterRing + sizeof(float) * a.hg * kD + (size_t)a.cap * 4 * (kCluster + 1);
            return run("page_select", bf ? k_page_select<__nv_bfloat16> : k_page_select<__half>,
                       dim3((unsigned)cluster_ctas(a)), kThreads, smem, kCluster);
        }
        a.hgroups = (a.p.Hkv + kHeads - 1) / kHeads;
        a.hg = (a.p.Hkv + a.hgroups - 1) / a.hgroups;
        const vsa_status e = run("page_scores", bf ? k_page_scores<__nv_bfloat16> : k_page_scores<__half>,
                                 dim3(kCtasSel), kThreads, kSmemSel, 1);
        if (e != VSA_OK) return e;
    }
    const dim3 rows((unsigned)(a.p.B * a.p.Hkv));
    return a.p.max_pages > kLongRow ? run("page_topk", k_page_topk<2 * kTopkThreads>, rows, 2 * kTopkThreads, 0, 1)
                                    : run("page_topk", k_page_topk<kTopkThreads>, rows, kTopkThreads, 0, 1);
}
