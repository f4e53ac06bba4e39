// paged_select.cu -- the pages each key/value head attends to, by the score
// of their mean key against the group's query (vsa_page_select).
//
// One launch. A cluster of 8 CTAs has one sequence and up to 8 key/value
// heads; the pages that compete (all but the first keep_first and the last
// keep_last) are cut into 8 runs, one per CTA. A CTA reads the fp32 means of
// its run once (8 lanes per page, 16 bytes per load; the heads of a page are
// neighbours in memory) and leaves an order-preserving 32-bit key per page
// and head in its shared memory. Then each CTA finishes one head: it reads
// the 8 CTAs' keys through the cluster's distributed shared memory and finds
// the last page to take under (key desc, page asc), 11 bits of (key, page)
// at a time from the top (a 2,048-bin histogram), until the bin that holds
// it is small enough to rank outright; then lists the taken pages in order.
// The scores never leave the SMs. The means stream through a ring of
// asynchronous copies per warp; a lane reads back what it copied itself.
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
    int hg, hgroups;  // heads per cluster, clusters per sequence
    int cap;          // pages per CTA at most
};

constexpr int kCluster = 8;
constexpr int kThreads = 256, kWarpsSel = kThreads / 32;
constexpr int kRing = 4;     // ring stages per warp, each four pages' means of one head (2 KB)
constexpr int kBins = 2048;
constexpr int kRank = 256;   // a bin of up to this many pages is ranked outright
constexpr int kIndexBits = 22;
constexpr int kRingBytes = kRing * 2048;
constexpr int kMaxSmem = 200 * 1024;  // dynamic, beside the bins and the list

// Shared memory of the rings, and later of one head's keys.
__host__ __device__ __forceinline__ int front_bytes(int cap) {
    const int ring = kWarpsSel * kRingBytes, keys = kCluster * cap * 4;
    return ring > keys ? ring : (keys + 15) & ~15;
}

// Larger score, larger key; -0 folded into +0, NaN counted as -inf.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) x = -INFINITY;
    if (x == 0.f) x = 0.f;
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Sum of the group's 16-bit queries at one dim: the fp32 running sum with
// its rounding errors kept aside (each found exactly), added at the end.
template <typename T> __device__ __forceinline__ float group_sum(const T *q, int G) {
    float s = to_f<T>(q[0]), err = 0.f;
    for (int m = 1; m < G; ++m) {
        const float x = to_f<T>(q[(long long)m * kD]);
        const float t = __fadd_rn(s, x), y = __fsub_rn(t, s);
        err = __fadd_rn(err, __fadd_rn(__fsub_rn(s, __fsub_rn(t, y)), __fsub_rn(x, y)));
        s = t;
    }
    return isfinite(s) ? __fadd_rn(s, err) : s;
}

// (key, page) as one number, the larger the better: 32 key bits, then the
// page counted from the end.
__device__ __forceinline__ uint64_t rank_of(uint32_t key, int c) {
    return ((uint64_t)key << kIndexBits) | (uint32_t)((1 << kIndexBits) - 1 - c);
}

template <typename T> __global__ void __launch_bounds__(kThreads) k_page_select(SelectArgs a) {
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ int hist[kBins];
    __shared__ int wsum[kWarpsSel];
    __shared__ int s_bin, s_above, s_in, s_fill;
    __shared__ uint64_t s_cut;
    __shared__ uint64_t list[kRank];
    uint32_t *mine = reinterpret_cast<uint32_t *>(sm);                   // [kCluster * cap] all keys of one head,
                                                                         // where the rings were
    float *sq = reinterpret_cast<float *>(sm + front_bytes(a.cap));      // [hg][128] summed queries
    uint32_t *keys = reinterpret_cast<uint32_t *>(sq + a.hg * kD);       // [hg][cap] keys of this CTA's run
    int *ids = reinterpret_cast<int *>(keys + (size_t)a.hg * a.cap);     // [cap] page ids of the run
    const Paged &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = (int)ptx::cluster_rank(), cl = (int)blockIdx.x / kCluster;
    const int b = cl / a.hgroups, h0 = (cl % a.hgroups) * a.hg, hn = min(a.hg, p.Hkv - h0);
    grid_wait();
    grid_go();
    const int len = paged_len(p, b), pages = (len + p.page - 1) >> p.page_log2;
    if (pages <= a.topk) {  // all of them: the same for every CTA of the cluster
        for (int hh = rank; hh < hn; hh += kCluster) {
            const long long row = (long long)b * p.Hkv + h0 + hh;
            for (int n = tid; n < a.topk; n += kThreads) a.idx[row * a.topk + n] = n < pages ? n : -1;
            if (tid == 0) a.cnt[row] = pages;
        }
        return;
    }
    // Competing pages c = j - first, 0 <= c < comp: every one is full, since the partial page is the last.
    const int comp = pages - a.first - a.last, take = a.topk - a.first - a.last;
    const int run = (comp + kCluster - 1) / kCluster;
    const int c0 = min(rank * run, comp), nc = min(run, comp - c0);

    for (int c = tid; c < nc; c += kThreads) ids[c] = paged_id(p, b, a.first + c0 + c);
    const T *q = static_cast<const T *>(a.q) + b * a.qs + (long long)h0 * p.G * kD;
    for (int e = tid; e < hn * kD; e += kThreads)
        sq[e] = group_sum<T>(q + (long long)(e / kD) * p.G * kD + e % kD, p.G);
    __syncthreads();

    // An item is four pages of one head; lane j of eight holds dims 32 i + 4 j + c of a page.
    const int sub = lane >> 3, j = lane & 7, items = (nc + 3) / 4 * hn;
    const uint32_t ring = ptx::smem_addr(sm) + wid * kRingBytes + lane * 16;
    auto copy = [&](int it, int stage) {
        const int hh = it % hn, c = it / hn * 4 + sub;
        const int id = c < nc ? ids[c] : -1;
        const float *src = a.mean + ((long long)max(id, 0) * p.Hkv + h0 + hh) * kD + 4 * j;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ring + stage * 2048 + i * 512),
                         "l"(src + 32 * i), "r"(id >= 0 ? 16 : 0)
                         : "memory");
    };
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s) {
        if (wid + s * kWarpsSel < items) copy(wid + s * kWarpsSel, s);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (int n = 0; wid + n * kWarpsSel < items; ++n) {
        const int it = wid + n * kWarpsSel, hh = it % hn, c = it / hn * 4 + sub;
        const int ahead = it + (kRing - 1) * kWarpsSel;
        if (ahead < items) copy(ahead, (n + kRing - 1) % kRing);  // the stage this lane read last
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        float x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 g = *reinterpret_cast<const float4 *>(sq + hh * kD + 32 * i + 4 * j);
            const float4 m = *reinterpret_cast<const float4 *>(sm + wid * kRingBytes + (n % kRing) * 2048 + i * 512 +
                                                               lane * 16);
            x[i][0] = __fmul_rn(g.x, m.x);
            x[i][1] = __fmul_rn(g.y, m.y);
            x[i][2] = __fmul_rn(g.z, m.z);
            x[i][3] = __fmul_rn(g.w, m.w);
        }
        // 128 -> 64 -> 32: dims 64 and 32 apart; then neighbours
        float y[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) y[d] = __fadd_rn(__fadd_rn(x[0][d], x[2][d]), __fadd_rn(x[1][d], x[3][d]));
        float r = __fadd_rn(__fadd_rn(y[0], y[1]), __fadd_rn(y[2], y[3]));
        r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 1));
        r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 2));
        r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 4));
        if (j == 0 && c < nc) keys[hh * a.cap + c] = order_key(ids[c] >= 0 ? r : -INFINITY);
    }
    ptx::cluster_sync();  // every run's keys are there

    for (int hh = rank; hh < hn; hh += kCluster) {
        const long long row = (long long)b * p.Hkv + h0 + hh;
        int *idx = a.idx + row * a.topk;
        const uint32_t base = ptx::smem_addr(keys + (size_t)hh * a.cap);
        // the head's keys from all runs, in page order
#pragma unroll
        for (int r = 0; r < kCluster; ++r) {
            const uint32_t at = ptx::cluster_addr(base, r);
            const int n = min(run, comp - r * run);
            for (int c = tid; c < n; c += kThreads) mine[r * run + c] = ld_cluster(at + 4 * c);
        }
        __syncthreads();
        auto each = [&](auto f) {
            for (int c = tid; c < comp; c += kThreads) f(rank_of(mine[c], c));
        };
        // cut: the `take`-th largest rank (ranks are distinct); 2^54 when none is taken
        uint64_t cut = 1ull << (32 + kIndexBits), prefix = 0;
        int rem = take, top = 32 + kIndexBits;  // bits [top, 54) of the cut are `prefix`
        while (rem > 0) {
            const int shift = max(top - 11, 0), bits = top - shift;
            for (int e = tid; e < kBins; e += kThreads) hist[e] = 0;
            __syncthreads();
            each([&](uint64_t k) {
                if (k >> top == prefix) atomicAdd(&hist[(int)((k >> shift) & ((1u << bits) - 1u))], 1);
            });
            __syncthreads();
            // thread t: bins 2047 - 8 t down to 2040 - 8 t
            int cnt[kBins / kThreads], sum = 0;
#pragma unroll
            for (int e = 0; e < kBins / kThreads; ++e) sum += cnt[e] = hist[kBins - 1 - tid * (kBins / kThreads) - e];
            int inc = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += y;
            }
            if (lane == 31) wsum[wid] = inc;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWarpsSel; ++w) inc += w < wid ? wsum[w] : 0;
            int above = inc - sum;  // pages in larger bins
            if (above < rem && inc >= rem) {
#pragma unroll
                for (int e = 0; e < kBins / kThreads; ++e)
                    if (above < rem) {
                        s_bin = kBins - 1 - tid * (kBins / kThreads) - e;
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
                    if (k >> top == prefix) list[atomicAdd(&s_fill, 1)] = k;
                });
                __syncthreads();
                if (tid < in) {
                    const uint64_t k = list[tid];
                    int larger = 0;
                    for (int e = 0; e < in; ++e) larger += list[e] > k ? 1 : 0;
                    if (larger == rem - 1) s_cut = k;
                }
                __syncthreads();
                cut = s_cut;
                break;
            }
            __syncthreads();  // s_bin and the bins are read before the next digit
        }
        // pages at or above the cut, in order: each warp has a contiguous share
        const int share = ((comp + kWarpsSel - 1) / kWarpsSel + 31) & ~31;
        const int lo = min(wid * share, comp), hi = min(lo + share, comp);
        auto chosen = [&](int c) { return rank_of(mine[c], c) >= cut; };
        int n = 0;
        for (int c = lo + lane; c - lane < hi; c += 32) n += __popc(__ballot_sync(0xffffffffu, c < hi && chosen(c)));
        __syncthreads();  // wsum was read
        if (lane == 0) wsum[wid] = n;
        __syncthreads();
        int at = a.first;
#pragma unroll
        for (int w = 0; w < kWarpsSel; ++w) at += w < wid ? wsum[w] : 0;
        for (int c = lo + lane; c - lane < hi; c += 32) {
            const bool on = c < hi && chosen(c);
            const unsigned m = __ballot_sync(0xffffffffu, on);
            if (on) idx[at + __popc(m & ((1u << lane) - 1u))] = a.first + c;
            at += __popc(m);
        }
        for (int e = tid; e < a.first; e += kThreads) idx[e] = e;
        for (int e = tid; e < a.last; e += kThreads) idx[a.topk - a.last + e] = pages - a.last + e;
        if (tid == 0) a.cnt[row] = a.topk;
        __syncthreads();  // the bins and sums serve the next head
    }
    ptx::cluster_sync();  // no CTA leaves while another reads its keys
}

}  // namespace
}  // namespace vsa

extern "C" vsa_status vsa_page_select(const vsa_paged_desc *desc, const void *q, int64_t q_stride,
                                      const float *k_mean, int topk, int keep_first, int keep_last,
                                      int32_t *page_idx, int32_t *page_cnt, vsa_stream_t stream) {
    using namespace vsa;
    SelectArgs a{};
    const vsa_status st = to_paged(desc, &a.p, true);
    if (st != VSA_OK) return st;
    if (!token_stride(q_stride, a.p.Hq, &a.qs)) return VSA_ERR_SHAPE;
    if (keep_first < 0 || keep_last < 1 || topk < 1 || (long long)keep_first + keep_last > topk) return VSA_ERR_SHAPE;
    if (!q || !k_mean || !page_idx || !page_cnt) return VSA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_mean) || ((uintptr_t)page_idx | (uintptr_t)page_cnt) & 3u) return VSA_ERR_LAYOUT;
    a.q = q;
    a.mean = k_mean;
    a.topk = topk;
    a.first = keep_first;
    a.last = keep_last;
    a.idx = page_idx;
    a.cnt = page_cnt;
    // Heads per cluster: as many as still leave a CTA for every SM.
    a.hg = 8;
    while (a.hg > 1 && ((long long)a.p.B * ((a.p.Hkv + a.hg - 1) / a.hg) * kCluster < 152 || a.hg / 2 >= a.p.Hkv))
        a.hg /= 2;
    a.cap = (std::min(a.p.max_pages, 1 << kIndexBits) + kCluster - 1) / kCluster;
    auto bytes = [&] {
        return front_bytes(a.cap) + sizeof(float) * a.hg * kD + (size_t)a.cap * 4 * (a.hg + 1);
    };
    while (a.hg > 1 && bytes() > kMaxSmem) a.hg /= 2;
    if (a.p.max_pages > (1 << kIndexBits) || bytes() > kMaxSmem) return VSA_ERR_UNSUPPORTED;
    a.hgroups = (a.p.Hkv + a.hg - 1) / a.hg;
    const long long ctas = (long long)a.p.B * a.hgroups * kCluster;
    if (ctas > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool bf = a.p.dtype == T_BF16;
    const void *fn = bf ? (const void *)k_page_select<__nv_bfloat16> : (const void *)k_page_select<__half>;
    const cudaError_t ae = ensure_smem_limit(fn, kMaxSmem);
    if (ae != cudaSuccess) return status_from_cuda(ae);
    prof_begin("page_select", s);
    const cudaError_t e = launch_paged(bf ? k_page_select<__nv_bfloat16> : k_page_select<__half>, dim3((unsigned)ctas),
                                       kThreads, bytes(), kCluster, a, s);
    prof_end(s);
    return status_from_cuda(e);
}
