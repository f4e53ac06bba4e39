// paged_select.cu -- the pages each key/value head attends to, by the score
// of their mean key against the group's query (vsa_page_select).
//
// Two launches: k_page_scores reads each full page's fp32 mean once (8 lanes
// per page, 16 bytes per load) and writes an order-preserving 32-bit key per
// page; k_page_topk finds, per row, the topk-th largest key 8 bits at a time
// (a 256-bin histogram per digit) and lists every key above it plus the
// lowest-indexed ties, ascending.
#include <algorithm>

#include "paged.cuh"

namespace vsa {
namespace {

struct SelectArgs {
    Paged p;
    const void *q;
    long long qs;
    const float *mean;
    int topk, first, last;
    int *idx, *cnt;
    uint32_t *keys;  // [B * Hkv, max_pages]
};

constexpr int kChunk = 128;  // pages per CTA of the scoring pass

// Larger score, larger key; -0 folded into +0, NaN counted as -inf. No key
// reaches 0xFFFFFFFF, which marks the pages that are always chosen.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) x = -INFINITY;
    if (x == 0.f) x = 0.f;
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <typename T> __global__ void __launch_bounds__(256) k_page_scores(SelectArgs a) {
    const Paged &p = a.p;
    const int row = blockIdx.x, b = row / p.Hkv, h = row % p.Hkv;
    const int len = paged_len(p, b), full = len >> p.page_log2, pages = (len + p.page - 1) >> p.page_log2;
    if (pages <= a.topk) return;  // every page is chosen
    const int lane = threadIdx.x & 31, sub = lane >> 3, j = lane & 7;
    // lane j of 8 holds dims 32 i + 4 j + c of the group's summed query
    float g[4][4];
    const T *q = static_cast<const T *>(a.q) + b * a.qs + (long long)h * p.G * kD;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) g[i][c] = 0.f;
    if (p.G == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) g[i][c] = to_f<T>(q[32 * i + 4 * j + c]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                double sum = 0.0;  // exact for any group of 16-bit values of like size: the order does not matter
                for (int m = 0; m < p.G; ++m) sum += (double)to_f<T>(q[(long long)m * kD + 32 * i + 4 * j + c]);
                g[i][c] = (float)sum;
            }
    }
    uint32_t *keys = a.keys + (long long)row * p.max_pages;
    for (int c0 = blockIdx.y * kChunk; c0 < pages; c0 += gridDim.y * kChunk) {
        const int end = min(pages, c0 + kChunk);
        for (int n = c0 + (int)(threadIdx.x >> 5) * 4; n < end; n += 32) {
            const int pg = n + sub;
            const bool kept = pg < a.first || pg >= pages - a.last || pg >= full;
            const int id = pg < end && !kept ? paged_id(p, b, pg) : -1;
            float x[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 m = id >= 0 ? __ldg(reinterpret_cast<const float4 *>(
                                               a.mean + ((long long)id * p.Hkv + h) * kD + 32 * i + 4 * j))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
                x[i][0] = __fmul_rn(g[i][0], m.x);
                x[i][1] = __fmul_rn(g[i][1], m.y);
                x[i][2] = __fmul_rn(g[i][2], m.z);
                x[i][3] = __fmul_rn(g[i][3], m.w);
            }
            // 128 -> 64 -> 32: dims 64 and 32 apart; then neighbours
            float y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                y[c] = __fadd_rn(__fadd_rn(x[0][c], x[2][c]), __fadd_rn(x[1][c], x[3][c]));
            float r = __fadd_rn(__fadd_rn(y[0], y[1]), __fadd_rn(y[2], y[3]));
            r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 1));
            r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 2));
            r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 4));
            if (j == 0 && pg < end)
                keys[pg] = kept ? 0xFFFFFFFFu : (id >= 0 ? order_key(r) : order_key(-INFINITY));
        }
    }
}

__global__ void __launch_bounds__(256) k_page_topk(SelectArgs a) {
    const Paged &p = a.p;
    const int row = blockIdx.x, b = row / p.Hkv, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int len = paged_len(p, b), pages = (len + p.page - 1) >> p.page_log2;
    int *idx = a.idx + (long long)row * a.topk;
    const int take = min(a.topk, pages);
    if (tid == 0) a.cnt[row] = take;
    for (int n = take + tid; n < a.topk; n += 256) idx[n] = -1;
    if (pages <= a.topk) {
        for (int n = tid; n < pages; n += 256) idx[n] = n;
        return;
    }
    __shared__ int hist[256];
    __shared__ int s_digit, s_above;
    __shared__ int wtot[8], wtie[8];
    const uint32_t *keys = a.keys + (long long)row * p.max_pages;
    uint32_t prefix = 0u, known = 0u;
    int rem = take;
    for (int shift = 24; shift >= 0; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        for (int n = tid; n < pages; n += 256) {
            const uint32_t key = keys[n];
            if ((key & known) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
        }
        __syncthreads();
        if (wid == 0) {  // lane l: digits 255 - 8 l down to 248 - 8 l
            int c[8], sum = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) sum += c[u] = hist[255 - 8 * lane - u];
            int inc = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += y;
            }
            int above = inc - sum;  // keys with a larger digit
            if (above < rem && inc >= rem) {
                int u = 0;
                while (above + c[u] < rem) above += c[u++];
                s_digit = 255 - 8 * lane - u;
                s_above = above;
            }
        }
        __syncthreads();
        rem -= s_above;
        prefix |= (uint32_t)s_digit << shift;
        known |= 255u << shift;
    }
    // every key above prefix, and the first `rem` keys equal to it, in order
    int done = 0, ties = 0;
    for (int n0 = 0; n0 < pages; n0 += 256) {
        const int n = n0 + tid;
        const uint32_t key = n < pages ? keys[n] : 0u;
        const bool tie = n < pages && key == prefix, over = n < pages && key > prefix;
        const unsigned mt = __ballot_sync(0xffffffffu, tie), lt = (1u << lane) - 1u;
        if (lane == 0) wtie[wid] = __popc(mt);
        __syncthreads();
        int before = ties, all = ties;
        for (int w = 0; w < 8; ++w) {
            before += w < wid ? wtie[w] : 0;
            all += wtie[w];
        }
        const bool on = over || (tie && before + __popc(mt & lt) < rem);
        const unsigned mo = __ballot_sync(0xffffffffu, on);
        if (lane == 0) wtot[wid] = __popc(mo);
        __syncthreads();
        int at = done, sum = done;
        for (int w = 0; w < 8; ++w) {
            at += w < wid ? wtot[w] : 0;
            sum += wtot[w];
        }
        if (on) idx[at + __popc(mo & lt)] = n;
        done = sum;
        ties = all;
    }
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
    const unsigned rows = (unsigned)(a.p.B * a.p.Hkv);
    if (a.p.max_pages > topk) {  // otherwise no row has anything to choose
        const unsigned chunks = (unsigned)std::min((a.p.max_pages + kChunk - 1) / kChunk, 65535);
        prof_begin("page_scores", s);
        if (a.p.dtype == T_BF16)
            k_page_scores<__nv_bfloat16><<<dim3(rows, chunks), 256, 0, s>>>(a);
        else
            k_page_scores<__half><<<dim3(rows, chunks), 256, 0, s>>>(a);
        prof_end(s);
        const vsa_status se = status_from_cuda(cudaGetLastError());
        if (se != VSA_OK) return se;
    }
    prof_begin("page_topk", s);
    k_page_topk<<<rows, 256, 0, s>>>(a);
    prof_end(s);
    return status_from_cuda(cudaGetLastError());
}
