// paged_attn.cuh -- attention of one token per sequence over a paged
// key/value cache (vsa_paged_attn, vsa_paged8_attn, vsa_paged_attn_weigh), all
// pages or the listed ones. kv below is the bits of a cached element: 16, or 8
// with a scale per block of 16 tokens (stream_blocks8).
//
//   O = sum_u W_u v_u / sum_u W_u,  LSE = max + log sum_u P_u,
//   P_u = exp(scale q.k_u - max), W_u = P_u rounded to the cache's 16 bits
//
// The products with V take 16-bit weights; O is divided by the sum of the
// weights it was made with, so these sum to one whatever the roundings did:
// keys of one score all round the same way, and the sum of the P_u left their
// common error in O (9,001 keys, scores 0 and -0.69, V = 1: 0.996 in bf16, and
// +inf in fp16 for V = 65504). What remains is u sum_u p_u |v_u - O|, u half a
// step of the type. The sum of the W_u comes from the same instruction, as the
// product with a column of ones: two more of a step's 64 (no time measured).
// The product of what the rounding leaves, P - W, would take 32 more: the error
// of random outputs falls from 1.1 to 1.2 times that of rounding them once to
// 1.0, and 16 sequences of up to 9,000 keys with 16 heads each go from 18.6 to
// 20.5 us, 64 of up to 16,000 from 83.7 to 84.9, 24 heads of 122,880 keys stay at
// 217; and 0 * inf would be NaN where an infinite value is attended. Not done.
//
// A segment is one (sequence, key/value head, chunk of up to 16 query heads
// of its group: one tile of the tensor instructions; a wider group's chunks
// read the same keys, from L2 but for the first); its keys, in the order of
// the pages attended, are cut into blocks of 16. A warp streams a run of
// blocks, two per step, through its own ring of asynchronous copies (a slot
// takes the 32 K rows of a step or its V rows, 256 bytes each, swizzled so that
// ldmatrix reads hit distinct banks; rows past a page's valid slots are filled
// with zeros, so whatever the cache holds there cannot reach the sums) and keeps its own running maximum, sum
// and output in registers: no warp waits for another while it streams. The
// products run on m16n8k16 tensor instructions with the group's query heads
// as rows. At one query token per sequence the kernel reads 512 bytes per
// 256 G multiply-adds, far to the memory side of the tensor cores' balance, so
// the instruction's rate does not bound it; the memory pipe does, and for
// short segments the chain of dependent loads before the first product.
//
// Short or equal segments: k_paged_attn_cluster, one launch. A segment is one
// cluster's (of 1 to 16 CTAs); the CTAs join their four warps' results in
// shared memory and send each row to the CTA that finishes it.
// Any lengths: k_paged_attn_runs. The blocks of all segments, end to end, are
// dealt to the grid's warps in equal contiguous runs, whatever the lengths of
// the batch: a CTA finds its run with one scan of the lengths, and each warp
// walks the segments of its own part of it. A segment inside one warp's run
// is finished there; where a CTA's whole run lies in one segment its warps'
// results are joined first; the remaining pieces of segments that cross runs
// go to the workspace (at most two per warp), and k_paged_join adds them in
// ascending order.
#pragma once

#include <algorithm>
#include <type_traits>

#include "e4m3.cuh"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace vsa {
namespace {

constexpr int kBlk = 16;        // keys per block; a warp takes two per step
constexpr int kRows = 16;       // query heads per segment at most
constexpr int kLead = 4;        // blocks a segment counts for beyond its own (its start-up time): 0, 1, 2, 3, 4
                                // measured 102, 92, 87, 85.1, 84.8 us on 64 sequences of 37 to 16,000 keys
// The same of an 8-bit cache, whose blocks stream in half the time: 4, 8, 12, 16 measured 81, 74.9, 75.5, 74.8 us on the
// same lengths.
constexpr int kLead8 = 8;
constexpr int kAlignedKeys = 1280;  // keys per CTA up to which segments of unknown lengths get a cluster each
// Of an 8-bit cache. Equal lengths, 4 heads per key head (us, clusters / runs), up to 800 keys per CTA: 1 head of 12,000
// keys 9.0 / 10.3, 8 of 8,000 8.9 / 10.3, 24 of 1,000 5.8 / 10.1, 64 of 2,400 11.6 / 13.6; more: 24 of 12,000 19.3 / 17.5,
// 8 of 16,000 13.7 / 12.8, 32 of 12,000 20.9 / 20.5, 64 of 8,000 28.1 / 31.1, 256 of 800 12.4 / 16.2 (unequal lengths would lose
// that: a cluster's longest decides). 16 heads per key head: 32 of 4,000 15.9 / 16.6, of 6,400 22.4 / 18.9, of 8,000 24.0 / 20.4.
constexpr int kAlignedKeys8 = 800;
constexpr int kFewCtas = 912;       // and CTAs in all, three at each place: 1,192 segments of 17 keys 11.6 us, 7.6 in runs;
                                    // 800 of 64 11.9, 14.2
constexpr int kAlignedCtas = 96;    // CTAs that nearly fill the memory pipe
constexpr int kMaxCluster = 16;     // 16,000 keys x 8 heads: 15.6 us, 22 with clusters of 8
constexpr int kWarps = 4;
constexpr int kStages = 3;      // ring slots per warp, for two CTAs per SM; five, where there are no more CTAs than SMs,
                                // left clusters of 16 without a place: 8 x 16,000 keys 15.7 -> 23 us
constexpr int kCtas = 304;      // two per SM on 152 SMs
constexpr int kStageBytes = 2 * kBlk * 256;  // the K or the V rows of a step
constexpr int kPitch = 136;     // floats per row of the warps' outputs in shared memory
template <int KV> constexpr int stage_bytes = KV == 8 ? kStageBytes / 2 : kStageBytes;
template <int KV> constexpr int smem_bytes = kWarps * kStages * stage_bytes<KV>;

struct AttnArgs {
    Paged p;
    const void *q;
    long long qs;
    const void *k, *v;
    const int *idx, *cnt;  // page lists (NULL: all pages)
    int cap;
    void *out;
    float *lse;
    int rc, rows;          // chunks of a group's heads, rows per chunk
    int cluster;           // CTAs per segment, one cluster; 0: equal runs of all segments' blocks
    int4 *seg;             // [segments] its pieces: first warp, warps before / CTAs joined / pieces in all
    float4 *ml;            // [2 * kCtas * kWarps, rows] maximum (of q.k), sum of P, sum of W, 0
    float *o;              // [2 * kCtas * kWarps, rows, 128]
    const float *ks, *vs;  // 8 bits: scales [num_pages, Hkv, page / 16]
    float2 *bw;            // vsa_paged_attn_weigh: [segments, blocks, rows] sum of P and the maximum of q.k it is relative
    int blocks;            // to; blocks a segment has room for
    float2 *stat;          // [B, Hq] a row's maximum of q.k and 1 / sum of P
};

// Keys of segment list entry n ((b) without page lists, (b, h) with): the
// positions it walks, valid or not.
__device__ __forceinline__ int seg_keys(const AttnArgs &a, int n) {
    if (!a.idx) return paged_len(a.p, n);
    return clampi(a.cnt[n], 0, a.cap) * a.p.page;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Copies the first `bytes` (0 or 16) and fills the rest with zeros.
__device__ __forceinline__ void cp16z(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void st_cluster4(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c += a b: a 16 x 16 (row), b 16 x 8 (col), fp32 accumulators.
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int seg_blocks(const AttnArgs &a, int n) { return (seg_keys(a, n) + kBlk - 1) / kBlk; }

// P's exponent per unit of q.k, in log2 units.
__device__ __forceinline__ float log2_scale(const AttnArgs &a) { return a.p.scale * kLog2e; }

// Where a segment's queries, keys and outputs are.
struct Segment {
    int bh, b, h;        // list row, sequence, key/value head
    int rows;            // query heads
    long long hq0;       // first (sequence, query head)
    long long id;        // list row and chunk
};
__device__ __forceinline__ Segment segment_of(const AttnArgs &a, int bh, int r) {
    const Paged &p = a.p;
    Segment s;
    s.bh = bh;
    s.b = bh / p.Hkv;
    s.h = bh % p.Hkv;
    s.rows = min(a.rows, p.G - r * a.rows);
    s.hq0 = (long long)s.b * p.Hq + s.h * p.G + r * a.rows;
    s.id = (long long)bh * a.rc + r;
    return s;
}

// Q as A fragments: row g (and g + 8), 8 k-steps; rows past the segment's are zero.
template <typename T> __device__ __forceinline__ void load_q(const AttnArgs &a, const Segment &sg, uint32_t (&qa)[8][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const T *qb = static_cast<const T *>(a.q) + (long long)sg.b * a.qs + (sg.hq0 - (long long)sg.b * a.p.Hq) * kD;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int row = g + 8 * e;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(qb + (long long)row * kD);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            qa[j][e] = row < sg.rows ? src[8 * j + t] : 0u;
            qa[j][2 + e] = row < sg.rows ? src[8 * j + 4 + t] : 0u;
        }
    }
}

// vsa_paged_attn_weigh: the sums of P (as lifted) over blocks blk and blk + 1 of
// a segment (those before `end`), each row's beside the maximum of q.k that it
// is relative to. The four lanes of a row add up: each ends with one
// (block, row) of the four.
__device__ __forceinline__ void store_weights(const AttnArgs &a, const Segment &sg, int blk, int end, const float (&sc)[4][4],
                                              float ref0, float ref1) {
    const int lane = threadIdx.x & 31, g = lane >> 2, e = lane & 1, h = (lane >> 1) & 1;
    float n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float v0 = (sc[2 * i][0] + sc[2 * i][1]) + (sc[2 * i + 1][0] + sc[2 * i + 1][1]);
        const float v1 = (sc[2 * i][2] + sc[2 * i][3]) + (sc[2 * i + 1][2] + sc[2 * i + 1][3]);
        n[i] = (e ? v1 : v0) + __shfl_xor_sync(0xffffffffu, e ? v0 : v1, 1);
    }
    const float sum = (h ? n[1] : n[0]) + __shfl_xor_sync(0xffffffffu, h ? n[0] : n[1], 2);
    const int row = g + 8 * e;
    if (row < sg.rows && blk + h < end)
        a.bw[(sg.id * a.blocks + blk + h) * a.rows + row] = make_float2(sum, e ? ref1 : ref0);
}

// One warp streams blocks [blk0, blk0 + nblk) of a segment, two at a time
// (32 keys: two independent chains of products, one maximum and one rescaling
// for both): the running maximum (of q.k), the sums of P and of W of rows
// g and g + 8, and their unnormalised outputs at dims 8 j + 2 t, + 1. The ring's slots take the
// K rows of a step, its V rows, the K rows of the next step and so on; two are
// in flight while one is used. The ring is free again afterwards.
template <typename T, bool kWeigh>
__device__ __forceinline__ void stream_blocks(const AttnArgs &a, const Segment &sg, const uint32_t (&qa)[8][4], int len,
                                              int blk0, int nblk, uint32_t ring, float (&m_run)[2], float (&l_run)[2],
                                              float (&w_run)[2], float (&acc)[16][4]) {
    const Paged &p = a.p;
    const int lane = threadIdx.x & 31, t = lane & 3, b = sg.b, bh = sg.bh;
    const T *K = static_cast<const T *>(a.k), *V = static_cast<const T *>(a.v);
    const float sl2 = log2_scale(a);
    constexpr float kLift = std::is_same<T, __half>::value ? 15.f : 0.f, kDrop = kLift != 0.f ? 0x1p-15f : 1.f;
    constexpr uint32_t kOnes = std::is_same<T, __half>::value ? 0x3C003C00u : 0x3F803F80u;
    const int key0 = blk0 * kBlk;
    // Window of up to 32 blocks, one per lane: the page (or -1), the slot in
    // it and the valid slots of the block.
    int w_id = -1, w_slot = 0, w_valid = 0, w_base = -32;
    auto window = [&](int i0) {
        w_base = i0;
        w_id = -1;
        w_valid = 0;
        if (i0 + lane < nblk) {
            const int pos = key0 + (i0 + lane) * kBlk;
            int j = pos >> p.page_log2;
            w_slot = pos & (p.page - 1);
            if (a.idx) j = (unsigned)j < (unsigned)a.cap ? a.idx[(long long)bh * a.cap + j] : -1;
            w_id = paged_id(p, b, j);
            if (w_id >= 0) w_valid = clampi(len - (j << p.page_log2) - w_slot, 0, kBlk);
        }
    };
    // A lane copies the 16-byte chunk lane % 16 of rows 2 e (lanes 0-15) and 2 e + 1 (16-31) of each block, stored at
    // chunk (lane % 16) ^ (row % 8).
    const long long lane_at = (long long)sg.h * p.head_stride + (lane >> 4) * p.tok_stride + 8 * (lane & 15);
    const uint32_t lane_dst = (lane >> 4) * 256 + (((lane & 15) ^ (lane >> 4)) << 4);
    const uint32_t two_rows = (uint32_t)p.tok_stride * 4;  // bytes
    long long at[2];  // of the step being copied: its blocks' elements in the cache, and their valid slots
    int ok[2];
    auto locate = [&](int step) {
        if (2 * step >= w_base + 32) window(2 * step);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int from = 2 * step + h - w_base;
            const int id = __shfl_sync(0xffffffffu, w_id, from);
            const int slot = __shfl_sync(0xffffffffu, w_slot, from);
            ok[h] = __shfl_sync(0xffffffffu, w_valid, from);
            // A block lies inside its page, so the address of a row without a token is the page's own too.
            at[h] = (long long)max(id, 0) * p.page_stride + slot * p.tok_stride + lane_at;
        }
    };
    auto copy = [&](const T *from, uint32_t slot) {
        const uint32_t dst = slot + lane_dst;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const char *src = reinterpret_cast<const char *>(from + at[h]);
            if (ok[h] == kBlk) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    cp16((dst + h * kBlk * 256 + e * 512) ^ ((2 * e & 7) << 4), src + (uint64_t)e * two_rows);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    cp16z((dst + h * kBlk * 256 + e * 512) ^ ((2 * e & 7) << 4), src + (uint64_t)e * two_rows,
                          2 * e + (lane >> 4) < ok[h] ? 16 : 0);
            }
        }
    };
    const int steps = (nblk + 1) / 2;
    uint32_t k_slot = ring, v_slot = ring + kStageBytes, free_slot = ring + 2 * kStageBytes;
    if (steps > 0) {
        locate(0);
        copy(K, k_slot);
        cp_commit();
        copy(V, v_slot);
        cp_commit();
    }

    m_run[0] = m_run[1] = -INFINITY;
    l_run[0] = l_run[1] = 0.f;
    float wsum[4] = {0.f, 0.f, 0.f, 0.f};  // rows g, g, g + 8, g + 8
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    for (int i = 0; i < steps; ++i) {
        const int live[2] = {ok[0], ok[1]};
        cp_wait<1>();
        __syncwarp();  // every lane's K copies have landed, and V of the step before was read
        if (i + 1 < steps) {
            locate(i + 1);
            copy(K, free_slot);
        }
        cp_commit();
        float sc[4][4];  // keys 8 u + 2 t, + 1 of rows g, g + 8
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[u][e] = 0.f;
        {
            // fragments a few products ahead of their use: f = 2 j + h is k-step j of block h
            constexpr int kAhead = 6;
            const int row = (lane & 7) + ((lane >> 4) << 3), c0 = (lane >> 3) & 1;
            uint32_t kb[kAhead][4];
            auto ld_k = [&](uint32_t (&r)[4], int f) {
                ldsm4(r, k_slot + ((f & 1) * kBlk + row) * 256 + (((f & ~1) + c0) ^ (row & 7)) * 16);
            };
#pragma unroll
            for (int f = 0; f < kAhead; ++f) ld_k(kb[f], f);
#pragma unroll
            for (int f = 0; f < 16; ++f) {
                mma16816<T>(sc[2 * (f & 1)], qa[f >> 1], kb[f % kAhead][0], kb[f % kAhead][1]);
                mma16816<T>(sc[2 * (f & 1) + 1], qa[f >> 1], kb[f % kAhead][2], kb[f % kAhead][3]);
                if (f + kAhead < 16) ld_k(kb[f % kAhead], f + kAhead);
            }
        }
        cp_wait<1>();
        __syncwarp();  // every lane's V copies have landed, and K of this step was read
        if (i + 1 < steps) copy(V, k_slot);
        cp_commit();
        constexpr int kAheadV = 6;
        const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8, vc0 = lane >> 4;
        uint32_t vb[kAheadV][4];
        auto ld_v = [&](uint32_t (&r)[4], int f) {  // f = 8 h + j: dims 16 j.. of block h
            ldsm4t(r, v_slot + ((f >> 3) * kBlk + vrow) * 256 + (((2 * (f & 7) + vc0) ^ (vrow & 7)) << 4));
        };
#pragma unroll
        for (int f = 0; f < kAheadV; ++f) ld_v(vb[f], f);  // to arrive while the softmax runs
        if (live[0] + live[1] < 2 * kBlk) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (8 * (u & 1) + 2 * t + (e & 1) >= live[u >> 1]) sc[u][e] = -INFINITY;
        }
        // running maximum m of the unscaled scores; P = 2^(scale log2(e) (s - m) + lift)
        float corr[2];
        bool moved = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mx = ptx::fmax3(sc[0][2 * e], sc[0][2 * e + 1], sc[1][2 * e]);
            mx = ptx::fmax3(mx, sc[1][2 * e + 1], sc[2][2 * e]);
            mx = ptx::fmax3(mx, sc[2][2 * e + 1], sc[3][2 * e]);
            mx = fmaxf(mx, sc[3][2 * e + 1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = ptx::fmax3(m_run[e], mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            moved = moved || mx != m_run[e];
            const float ref = mx == -INFINITY ? 0.f : mx;  // a row without keys so far
            corr[e] = ptx::ex2((m_run[e] - ref) * sl2);
            m_run[e] = mx;
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    // the difference first: scale * s by itself loses what lies below its own last bit
                    const float pr = ptx::ex2(fmaf(sc[u][2 * e + c] - ref, sl2, kLift));
                    sc[u][2 * e + c] = pr;
                    sum += pr;
                }
            l_run[e] = fmaf(l_run[e], corr[e], sum);  // this lane's keys; quads are joined at the end
        }
        if constexpr (kWeigh) store_weights(a, sg, blk0 + 2 * i, blk0 + nblk, sc, m_run[0], m_run[1]);
        if (__any_sync(0xffffffffu, moved)) {
            wsum[0] *= corr[0], wsum[1] *= corr[0], wsum[2] *= corr[1], wsum[3] *= corr[1];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                acc[j][0] *= corr[0];
                acc[j][1] *= corr[0];
                acc[j][2] *= corr[1];
                acc[j][3] *= corr[1];
            }
        }
        // W: P rounded to the cache's 16-bit type for the product with V; the sum of P, for the LSE, keeps the
        // unrounded values. fp16 has no full steps below 2^-14, and a long row's keys may all lie below that next to
        // one large score: there P is lifted into [0, 2^15], full steps down to 2^-29.
        uint32_t pa[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                pa[h][2 * u] = pack2<T>(sc[2 * h + u][0], sc[2 * h + u][1]);
                pa[h][2 * u + 1] = pack2<T>(sc[2 * h + u][2], sc[2 * h + u][3]);
            }
        mma16816<T>(wsum, pa[0], kOnes, kOnes);
        mma16816<T>(wsum, pa[1], kOnes, kOnes);
#pragma unroll
        for (int f = 0; f < 16; ++f) {
            mma16816<T>(acc[2 * (f & 7)], pa[f >> 3], vb[f % kAheadV][0], vb[f % kAheadV][1]);
            mma16816<T>(acc[2 * (f & 7) + 1], pa[f >> 3], vb[f % kAheadV][2], vb[f % kAheadV][3]);
            if (f + kAheadV < 16) ld_v(vb[f % kAheadV], f + kAheadV);
        }
        const uint32_t was_k = k_slot;
        k_slot = free_slot;
        free_slot = v_slot;
        v_slot = was_k;
    }
    cp_wait<0>();
    __syncwarp();  // the warp's ring is free
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 1);
        l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 2);
        l_run[e] *= kDrop;  // the outputs and the sum of W they are divided by stay lifted
        w_run[e] = wsum[2 * e];
    }
}

// ------------------------------------------------------------------ 8 bits
// The same walk over a cache of e4m3 bytes with a scale per block of 16 tokens
// and key/value head. Bytes become fp16 (exactly: e4m3 has 4 significant bits and
// exponents from -9 to 8), q becomes fp16 beside a power of two per row that
// brings its largest entry into [2^14, 2^15) (bf16's 8 significant bits fit fp16's
// 11 down to 2^-29 of that entry, below that to 2^-40 of it), and the products run
// on the fp16 instructions for both types. Their sums times the k scale and the row's
// power of two are the scores, q.k in fp32 as in the 16-bit walk (the power taken into the
// softmax scale instead, keys near 2^110 overflowed with queries as small, and rows near
// 2^-100 under a small softmax scale became NaN). The
// v scales multiply the weights: acc is kept relative to a power of two, and a
// block's weights are multiplied by its scale over that, exact as long as the
// product is a normal fp16 number, 2^-14 and more. The sum W of the rounded weights is
// taken before, so that the weights that O is made with sum to one as above.
// While all v scales of a warp's blocks lie within kSpan of each other the power of two is the
// largest one met (vrun), for all rows: the key of the largest weight, 2^14 by
// the lift, then has a product of 2^8 or more, and what the roundings of products
// below 2^-14 leave is 2^-33 of that per key. Scales further apart (`far`, looked at
// for 32 blocks at a time) would take that room away: a block of the largest
// scale that is hardly attended left the other weights a few bits or none. From there
// on each row has a power of two of its own, by its largest product of weight
// and scale: two more maxima per row and step, and the weights multiplied in
// fp32, in a loop apart, so that the common one has no branch for it (scales 2^20 apart:
// the batch below 75.0 us, the long context 119.7, 16 heads on each of 2, 16 sequences 19.3).
//
// At half the bytes per key the instructions count: keys and dims are the rows
// of the products here, the query heads their columns, NT tiles of 8. Up to 8
// heads (NT = 1) that is half of the 16-bit walk's products, exponentials and
// accumulators: 34 products, 128 conversions and 8 exponentials per thread and
// step of 32 keys. 24 heads of 122,880 keys (756 MB): 118 us, 94% of the measured
// copy rate (heads as rows, as in the 16-bit walk, 172 us); 64 sequences of 37 to
// 16,000 keys x 8 heads (385 MB) 73 us, 77%: the CTAs' start, a segment's first
// loads and the join are 10 of the rest. A warp alone takes about 1,480 cycles and 600
// instructions per step, one chain from the copies' wait to the products: left out
// one at a time, the copies are 18% of it, products, conversions, permutations and
// shuffles under 5% each (two fp32 divisions were 10%), so a few long rows gain little
// over 16 bits (one head of 30,000 keys 10.1 us; 16 heads on each of 2, 16 sequences
// of up to 9,000 keys 16.1, 14.5 in 16 bits, NT = 2). Two accumulators per product
// left all of these as they are, a third step in the ring made them 2 to 6% slower.
//   S^T (keys x heads) = K (16 keys x 16 dims) Q^T, O^T (dims x heads) = V^T (16 dims x 16 keys) P^T
// A row of 128 bytes is 8 chunks of 16, stored at chunk ^ (row % 8). Thread (g, t)
// reads bytes 32 t .. 32 t + 31 of keys g and g + 8 of a block and takes word j for
// k-step j: the order of the dims among the k-steps is free as long as Q's
// fragments have the same. V comes through transposing 16-bit loads: a word holds
// dims 2 g, 2 g + 1 of keys 2 t, 2 t + 1; a byte permutation and two conversions
// make it rows g and g + 8 of a tile, which so are the dims 2 g and 2 g + 1 of its
// 16. P^T is turned by movmatrix.

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Q as B fragments in fp16: head 8 n + g, k-step j at dims 32 t + 4 j .. + 3; qs: the powers of two of heads 8 n + 2 t + e.
template <typename T, int NT>
__device__ __forceinline__ void load_q8(const AttnArgs &a, const Segment &sg, uint32_t (&qb)[NT][8][2], float (&qs)[2 * NT]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const T *from = static_cast<const T *>(a.q) + (long long)sg.b * a.qs + (sg.hq0 - (long long)sg.b * a.p.Hq) * kD;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = 8 * n + g;
        uint4 x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            x[c] = row < sg.rows ? reinterpret_cast<const uint4 *>(from + (long long)row * kD + 32 * t)[c]
                                 : make_uint4(0, 0, 0, 0);
        uint32_t w[16] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w,
                          x[2].x, x[2].y, x[2].z, x[2].w, x[3].x, x[3].y, x[3].z, x[3].w};
        float down = 1.f;
        if constexpr (!std::is_same<T, __half>::value) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 v = unpack2<T>(w[i]);
                top = ptx::fmax3(top, fabsf(v.x), fabsf(v.y));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // top = 1.m 2^e: to 2^14; an infinite top keeps its products infinite
            const int e = top == 0.f ? 14 : clampi((int)(__float_as_uint(top) >> 23) - 127, -100, 127);
            const float up = power_of(14 - e);
            down = power_of(e - 14);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 v = unpack2<T>(w[i]);
                w[i] = pack2<__half>(v.x * up, v.y * up);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) qs[2 * n + e] = __shfl_sync(0xffffffffu, down, 4 * (2 * t + e));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            qb[n][j][0] = w[2 * j];
            qb[n][j][1] = w[2 * j + 1];
        }
    }
}

// store_weights for the turned scores: sc[block][8 n + ..] has keys g, g + 8 by heads 2 t, 2 t + 1. The eight lanes of a
// head add up; four of them end with one (block, head) each.
template <int NT>
__device__ __forceinline__ void store_weights8(const AttnArgs &a, const Segment &sg, int blk, int end,
                                               const float (&sc)[2][NT][4], const float (&ref)[2 * NT]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, e = g & 1, h = (g >> 1) & 1;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float v0 = sc[i][n][0] + sc[i][n][2], v1 = sc[i][n][1] + sc[i][n][3];
            s[i] = (e ? v1 : v0) + __shfl_xor_sync(0xffffffffu, e ? v0 : v1, 4);
        }
        float sum = (h ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, h ? s[0] : s[1], 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = 8 * n + 2 * t + e;
        if (g < 4 && row < sg.rows && blk + h < end)
            a.bw[(sg.id * a.blocks + blk + h) * a.rows + row] = make_float2(sum, e ? ref[2 * n + 1] : ref[2 * n]);
    }
}

// A score tile's weights in fp16, turned into the B operands of the products with V.
__device__ __forceinline__ void turn_weights(const float (&sc)[4], uint32_t (&pb)[2]) {
    pb[0] = turn8x8(pack2<__half>(sc[0], sc[1]));
    pb[1] = turn8x8(pack2<__half>(sc[2], sc[3]));
}
// Largest over smallest v scale up to which a warp's outputs are relative to one power of two for all rows (stream_blocks8).
constexpr float kSpan = 64.f;
// The smaller one, NaN if either is.
__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
// e of an x with |x| in [2^e, 2^(e + 1)), -126 at least.
__device__ __forceinline__ int exponent_of(float x) { return max((int)(__float_as_uint(x) >> 23 & 255), 1) - 127; }

// stream_blocks for 8 bits: m_run, l_run, w_run of heads 8 n + 2 t + e at 2 n + e, their outputs' dims 16 j + 2 g and + 1 in
// acc[8 n + j][e] and [2 + e], finished: divided by w, and scaled.
template <int NT, bool kWeigh>
__device__ __forceinline__ void stream_blocks8(const AttnArgs &a, const Segment &sg, const uint32_t (&qb)[NT][8][2],
                                               const float (&qs)[2 * NT], int len, int blk0, int nblk, uint32_t ring,
                                               float (&m_run)[2 * NT], float (&l_run)[2 * NT], float (&w_run)[2 * NT],
                                               float (&acc)[8 * NT][4]) {
    const Paged &p = a.p;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, b = sg.b, bh = sg.bh;
    const unsigned char *K = static_cast<const unsigned char *>(a.k), *V = static_cast<const unsigned char *>(a.v);
    const float sl2 = log2_scale(a);
    constexpr float kLift = 14.f, kDrop = 0x1p-14f;
    constexpr int kStage8 = stage_bytes<8>;
    constexpr uint32_t kOnes[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
    const int key0 = blk0 * kBlk;
    // Window of up to 32 blocks, one per lane: page (or -1), slot, valid slots and scales.
    int w_id = -1, w_slot = 0, w_valid = 0, w_base = -32;
    float w_ks = 0.f, w_vs = 0.f;
    auto window = [&](int i0) {
        w_base = i0;
        w_id = -1;
        w_valid = 0;
        w_ks = w_vs = 0.f;
        if (i0 + lane < nblk) {
            const int pos = key0 + (i0 + lane) * kBlk;
            int j = pos >> p.page_log2;
            w_slot = pos & (p.page - 1);
            if (a.idx) j = (unsigned)j < (unsigned)a.cap ? a.idx[(long long)bh * a.cap + j] : -1;
            w_id = paged_id(p, b, j);
            if (w_id >= 0) w_valid = clampi(len - (j << p.page_log2) - w_slot, 0, kBlk);
            if (w_valid > 0) {
                const long long at = ((long long)w_id * p.Hkv + sg.h) * (p.page / kBlk) + w_slot / kBlk;
                w_ks = a.ks[at];
                w_vs = a.vs[at];
            }
        }
    };
    // A lane copies the 16-byte chunk lane % 8 of rows 4 e + lane / 8 of each block.
    const long long lane_at = (long long)sg.h * p.head_stride + (lane >> 3) * p.tok_stride + 16 * (lane & 7);
    const uint32_t lane_dst = (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
    const uint32_t four_rows = (uint32_t)p.tok_stride * 4;
    long long at[2];
    int ok[2];
    auto locate = [&](int step) {
        if (2 * step >= w_base + 32) window(2 * step);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int from = 2 * step + h - w_base;
            const int id = __shfl_sync(0xffffffffu, w_id, from);
            const int slot = __shfl_sync(0xffffffffu, w_slot, from);
            ok[h] = __shfl_sync(0xffffffffu, w_valid, from);
            at[h] = (long long)max(id, 0) * p.page_stride + slot * p.tok_stride + lane_at;
        }
    };
    // The outputs are relative to vrun, the largest power of two met and 2^126 at most (vnext: with the window's scales); once
    // far, each row's to 2^exp_of(peak): its largest product of (lifted) weight and scale so far as a logarithm, not rounded,
    // since it falls with the weights by less than a binade per step. Every lane keeps a copy for its rows.
    __shared__ float s_peak[kWarps][2 * NT][32];
    float(&peak)[2 * NT][32] = s_peak[threadIdx.x >> 5];
    auto exp_of = [](float x) { return clampi((int)floorf(x) - 12, -300, 300); };
    float vrun = 0x1p-126f, vnext = vrun, vlow = INFINITY;
    bool far = false;
    float ksc[2], vsc[2];
    auto scales = [&](int step) {  // of the step located last
        if (2 * step == w_base) {  // a window's first: all of its scales; those of 0 (no tokens) do not count
            const uint32_t u = __float_as_uint(w_vs) & 0x7fffffffu;
            const uint32_t top = min(__reduce_max_sync(0xffffffffu, u), 0x7e800000u);  // 2^126
            vlow = fminf(vlow, __uint_as_float(__reduce_min_sync(0xffffffffu, u ? u : 0x7f800000u)));
            vnext = fmaxf(vrun, __uint_as_float(top & 0x7f800000u));
            far = far || vnext > kSpan * vlow;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int from = 2 * step + h - w_base;
            ksc[h] = __shfl_sync(0xffffffffu, w_ks, from);
            vsc[h] = __shfl_sync(0xffffffffu, w_vs, from);
        }
    };
    auto copy = [&](const unsigned char *from, uint32_t slot) {
        const uint32_t dst = slot + lane_dst;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const unsigned char *src = from + at[h];
            if (ok[h] == kBlk) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    cp16((dst + h * kBlk * 128 + e * 512) ^ ((e & 1) << 6), src + (uint64_t)e * four_rows);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    cp16z((dst + h * kBlk * 128 + e * 512) ^ ((e & 1) << 6), src + (uint64_t)e * four_rows,
                          4 * e + (lane >> 3) < ok[h] ? 16 : 0);
            }
        }
    };
    const int steps = (nblk + 1) / 2;
    uint32_t k_slot = ring, v_slot = ring + kStage8, free_slot = ring + 2 * kStage8;
    if (steps > 0) {
        locate(0);
        copy(K, k_slot);
        cp_commit();
        copy(V, v_slot);
        cp_commit();
        scales(0);
    }

    float wsum[NT][4];
#pragma unroll
    for (int e = 0; e < 2 * NT; ++e) m_run[e] = -INFINITY, l_run[e] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) wsum[n][e] = 0.f;
#pragma unroll
    for (int j = 0; j < 8 * NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    auto step = [&](auto is_far, int i) {
        constexpr bool kFar = decltype(is_far)::value;
        const int live[2] = {ok[0], ok[1]};
        cp_wait<1>();
        __syncwarp();  // every lane's K copies have landed, and V of the step before was read
        if (i + 1 < steps) {
            locate(i + 1);
            copy(K, free_slot);
        }
        cp_commit();
        float sc[2][NT][4];  // block h: keys g, g, g + 8, g + 8 by heads 8 n + 2 t, + 1, ..
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[h][n][e] = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // bytes 32 t + 16 half ..
            uint4 kw[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) kw[u] = lds16(k_slot + (8 * u + g) * 128 + (((2 * t + half) ^ g) << 4));
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 &x = kw[2 * h], &y = kw[2 * h + 1];
                    const uint32_t lo = j == 0 ? x.x : j == 1 ? x.y : j == 2 ? x.z : x.w;
                    const uint32_t hi = j == 0 ? y.x : j == 1 ? y.y : j == 2 ? y.z : y.w;
                    const uint32_t ka[4] = {half2_of(lo), half2_of(hi), half2_of(lo >> 16), half2_of(hi >> 16)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16816<__half>(sc[h][n], ka, qb[n][4 * half + j][0], qb[n][4 * half + j][1]);
                }
        }
        cp_wait<1>();
        __syncwarp();  // every lane's V copies have landed, and K of this step was read
        if (i + 1 < steps) copy(V, k_slot);
        cp_commit();
        const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8, vc0 = lane >> 4;
        uint32_t vb[8][4];
#pragma unroll
        for (int f = 0; f < 8; ++f)  // f = 4 h + j: dims 32 j .. of block h
            ldsm4t(vb[f], v_slot + ((f >> 2) * kBlk + vrow) * 128 + (((2 * (f & 3) + vc0) ^ (vrow & 7)) << 4));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[h][n][e] *= min_nan(ksc[h] * qs[2 * n + (e & 1)], 0x1p127f);
        if (live[0] + live[1] < 2 * kBlk) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (g + 8 * (e >> 1) >= live[h]) sc[h][n][e] = -INFINITY;
        }
        // A block's ratio to vrun is below 2 (of larger scales than 2^126 4, and 2^14 times that is still in fp16).
        float ratio[2] = {1.f, 1.f}, vcorr = 1.f;
        if constexpr (!kFar) {
            const float inv = __uint_as_float(0x7f000000u - __float_as_uint(vnext));  // of a power of two
            vcorr = vrun * inv;
            vrun = vnext;
            ratio[0] = vsc[0] * inv;
            ratio[1] = vsc[1] * inv;
        }
        float corr[2 * NT];
        bool moved = vcorr != 1.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * n + e;
                float mx = fmaxf(ptx::fmax3(sc[0][n][e], sc[0][n][2 + e], sc[1][n][e]), sc[1][n][2 + e]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = ptx::fmax3(m_run[r], mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                moved = moved || mx != m_run[r];
                const float ref = mx == -INFINITY ? 0.f : mx;  // a row without keys so far
                corr[r] = ptx::ex2((m_run[r] - ref) * sl2);
                m_run[r] = mx;
                float sum = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float pr = ptx::ex2(fmaf(sc[h][n][2 * c + e] - ref, sl2, kLift));
                        sc[h][n][2 * c + e] = pr;
                        sum += pr;
                    }
                l_run[r] = fmaf(l_run[r], corr[r], sum);  // this lane's keys; the eight of a head are joined at the end
            }
        if constexpr (kWeigh) store_weights8<NT>(a, sg, blk0 + 2 * i, blk0 + nblk, sc, m_run);
        if constexpr (kFar) {
            // The sum of the weights as below; then the weights for the outputs: a row's largest product of weight and scale
            // so far comes to [2^12, 2^14) (a scale of 2^127: a binade more), and the outputs with it.
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                wsum[n][0] *= corr[2 * n], wsum[n][1] *= corr[2 * n + 1];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[2];
                    turn_weights(sc[h][n], w);
                    mma16816<__half>(wsum[n], kOnes, w[0], w[1]);
                }
            }
            int lv[2];
            float part[2];  // a scale is part 2^lv
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                lv[h] = min(exponent_of(vsc[h]), 126);
                part[h] = vsc[h] * power_of(-lv[h]);
            }
#pragma unroll
            for (int r = 0; r < 2 * NT; ++r) {
                const int n = r >> 1, e = r & 1;
                const float before = peak[r][lane];
                float now = corr[r] > 0.f ? before + __log2f(corr[r]) : -INFINITY;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float top = fmaxf(sc[h][n][e], sc[h][n][2 + e]);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    if (top > 0.f && vsc[h] != 0.f) now = fmaxf(now, (float)(exponent_of(top) + lv[h]));
                }
                if (now == -INFINITY) now = before;
                peak[r][lane] = now;
                const int to = exp_of(now);
                const float by = corr[r] * power_of(clampi(exp_of(before) - to, -126, 127));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[8 * n + j][e] *= by;
                    acc[8 * n + j][2 + e] *= by;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // in two factors: a small weight's may be 2^138
                    const int up = clampi(lv[h] - to, -252, 252), one = up >> 1;
                    const float f1 = power_of(one), f2 = power_of(up - one) * part[h];
                    sc[h][n][e] = sc[h][n][e] * f1 * f2;
                    sc[h][n][2 + e] = sc[h][n][2 + e] * f1 * f2;
                }
            }
        } else if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                wsum[n][0] *= corr[2 * n], wsum[n][1] *= corr[2 * n + 1];
                const float c0 = corr[2 * n] * vcorr, c1 = corr[2 * n + 1] * vcorr;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[8 * n + j][0] *= c0;
                    acc[8 * n + j][1] *= c1;
                    acc[8 * n + j][2] *= c0;
                    acc[8 * n + j][3] *= c1;
                }
            }
        }
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                turn_weights(sc[h][n], pb[h][n]);
                if constexpr (!kFar) mma16816<__half>(wsum[n], kOnes, pb[h][n][0], pb[h][n][1]);
            }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (!kFar && ratio[h] != 1.f) {  // the same for the whole warp
                const __half2 by = __float2half2_rn(ratio[h]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const __half2 x = __hmul2(*reinterpret_cast<__half2 *>(&pb[h][n][u]), by);
                        pb[h][n][u] = *reinterpret_cast<const uint32_t *>(&x);
                    }
            }
#pragma unroll
        for (int f = 0; f < 8; ++f)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint32_t lo = __byte_perm(vb[f][2 * c], 0, 0x3120), hi = __byte_perm(vb[f][2 * c + 1], 0, 0x3120);
                const uint32_t va[4] = {half2_of(lo), half2_of(lo >> 16), half2_of(hi), half2_of(hi >> 16)};
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma16816<__half>(acc[8 * n + 2 * (f & 3) + c], va, pb[f >> 2][n][0], pb[f >> 2][n][1]);
            }
        const uint32_t was_k = k_slot;
        k_slot = free_slot;
        free_slot = v_slot;
        v_slot = was_k;
        if (i + 1 < steps) scales(i + 1);
    };
    int i = 0;
    for (; i < steps && !far; ++i) step(std::false_type{}, i);
    if (far) {
#pragma unroll
        for (int r = 0; r < 2 * NT; ++r) peak[r][lane] = (float)(exponent_of(vrun) + 12);
        for (; i < steps; ++i) step(std::true_type{}, i);
#pragma unroll
        for (int r = 0; r < 2 * NT; ++r) {  // finished here: over w, times 2^e in three factors, -300 <= e <= 300
            const float w = wsum[r >> 1][r & 1], inv = w == 0.f ? 0.f : 1.f / w;
            const int e = exp_of(peak[r][lane]), e1 = e / 3, e2 = (e - e1) / 2;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float &x = acc[8 * (r >> 1) + j][2 * c + (r & 1)];
                    x = x * inv * power_of(e1) * power_of(e2) * power_of(e - e1 - e2);
                }
        }
        vrun = 1.f;
    }
    cp_wait<0>();
    __syncwarp();  // the warp's ring is free
#pragma unroll
    for (int r = 0; r < 2 * NT; ++r) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], off);
        l_run[r] *= kDrop;
        w_run[r] = wsum[r >> 1][r & 1];
        const float inv = far ? 1.f : w_run[r] == 0.f ? 0.f : 1.f / w_run[r];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float &x = acc[8 * (r >> 1) + j][2 * c + (r & 1)];
                x = x * inv * vrun;
            }
    }
}

// Where a warp's results of a segment are: NT = 0 is the 16-bit walk, 1 and 2 the 8-bit one's tiles of heads.
template <int NT> struct Frag {
    static constexpr bool k8 = NT > 0;
    static constexpr int kv = k8 ? 8 : 16, R = k8 ? 2 * NT : 2, A = k8 ? 8 * NT : 16;
    static __device__ __forceinline__ int row(int r) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        return k8 ? 8 * (r >> 1) + 2 * t + (r & 1) : g + 8 * r;
    }
    // one of the lanes that hold row(r)'s sums
    static __device__ __forceinline__ bool tells() { return k8 ? (threadIdx.x & 31) < 4 : (threadIdx.x & 3) == 0; }
    // f(d, x) for a thread's parts x of row(r), at dims d and d + 1
    template <typename F> static __device__ __forceinline__ void each(const float (&acc)[A][4], int r, F f) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        if constexpr (k8) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f(16 * j + 2 * g, make_float2(acc[8 * (r >> 1) + j][r & 1], acc[8 * (r >> 1) + j][2 + (r & 1)]));
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) f(8 * j + 2 * t, make_float2(acc[j][2 * r], acc[j][2 * r + 1]));
        }
    }
};
// The queries, and the walk with them.
template <typename T, int NT, bool kWeigh>
__device__ __forceinline__ void attend_blocks(const AttnArgs &a, const Segment &sg, int len, int blk0, int nblk, uint32_t ring,
                                              float (&m_run)[Frag<NT>::R], float (&l_run)[Frag<NT>::R],
                                              float (&w_run)[Frag<NT>::R], float (&acc)[Frag<NT>::A][4]) {
    if constexpr (NT > 0) {
        uint32_t qb[NT][8][2];
        float qs[2 * NT];
        load_q8<T, NT>(a, sg, qb, qs);
        stream_blocks8<NT, kWeigh>(a, sg, qb, qs, len, blk0, nblk, ring, m_run, l_run, w_run, acc);
    } else {
        uint32_t qa[8][4];
        load_q<T>(a, sg, qa);
        stream_blocks<T, kWeigh>(a, sg, qa, len, blk0, nblk, ring, m_run, l_run, w_run, acc);
    }
}

// What a piece with maximum m weighs beside one with maximum `ref`. The
// difference first, as within a piece: scaled maxima are rounded, by more than
// what is between two large ones (of 8 million: up to a factor of two in the
// weights), and with the largest softmax scales they are infinite.
__device__ __forceinline__ float beside(float m, float ref, float sl2) { return ptx::ex2((m - ref) * sl2); }

// What a piece's output counts for in a join beyond its maximum: unnormalised
// outputs hold their weights, finished ones (8 bits) do not.
template <int KV> __device__ __forceinline__ float own_weight(float w) { return KV == 8 ? w : 1.f; }

// Joins the CTA's four warps: stat(row, {M, l, w, 0}) once per row, with the
// maximum M and the sums l of P and w of W, then out(row, o) per
// row, in one warp, with a lane's dims 4 lane..: the unnormalised output, or
// where `done`, and always of an 8-bit cache, the finished one (divided by w).
// The rows' weights come first, side by side: one after another, with the
// division and the logarithm of each, 16 rows took 2.4 us more than 5.
// The warps' rings hold the outputs meanwhile.
template <int NT, typename S, typename F>
__device__ __forceinline__ void join_warps(unsigned char *smem, int rows, float sl2, const float (&m_run)[Frag<NT>::R],
                                           const float (&l_run)[Frag<NT>::R], const float (&w_run)[Frag<NT>::R],
                                           const float (&acc)[Frag<NT>::A][4], bool done, S stat, F out) {
    constexpr int KV = Frag<NT>::kv;
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows], s_w[kWarps][kRows], s_f[kWarps][kRows];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    float *so = reinterpret_cast<float *>(smem + wid * kStages * stage_bytes<KV>);
#pragma unroll
    for (int r = 0; r < Frag<NT>::R; ++r) {
        const int row = Frag<NT>::row(r);
        if (Frag<NT>::tells()) {
            s_m[wid][row] = m_run[r];
            s_l[wid][row] = l_run[r];
            s_w[wid][row] = w_run[r];
        }
        if (row < rows)
            Frag<NT>::each(acc, r, [&](int d, float2 x) { *reinterpret_cast<float2 *>(so + row * kPitch + d) = x; });
    }
    __syncthreads();
    if (tid < kWarps * kRows) {  // the warps' weights
        const int mine = tid / kRows, row = tid % kRows;
        float M = -INFINITY, l = 0.f, w = 0.f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) M = fmaxf(M, s_m[v][row]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
            const float f = beside(s_m[v][row], ref, sl2);
            l += f * s_l[v][row];
            w += f * s_w[v][row];
        }
        const float f = beside(s_m[mine][row], ref, sl2) * own_weight<KV>(s_w[mine][row]);
        s_f[mine][row] = !(done || KV == 8) ? f : w == 0.f ? 0.f : f / w;
        if (mine == 0 && row < rows) stat(row, make_float4(M, l, w, 0.f));
    }
    __syncthreads();
#pragma unroll 2
    for (int row = wid; row < rows; row += kWarps) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = s_f[w][row];
            const float *from = reinterpret_cast<const float *>(smem + w * kStages * stage_bytes<KV>);
            const float4 x = *reinterpret_cast<const float4 *>(from + row * kPitch + 4 * lane);
            o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
        }
        out(row, o);
    }
}
template <typename T> __device__ __forceinline__ uint2 pack4(float4 o) {
    return make_uint2(pack2<T>(o.x, o.y), pack2<T>(o.z, o.w));
}
// A finished row's LSE; where pages are weighed also its maximum and sum, which the LSE is too short for (rounded, it is off
// by 2^-24 of itself, and weights by a factor of e to that: a hundredth for scores of 100,000, anything for 1e9).
__device__ __forceinline__ void store_row(const AttnArgs &a, long long row, float M, float l, float sl2) {
    a.lse[row] = l == 0.f ? -INFINITY : kLn2 * __fadd_rn(__fmul_rn(M, sl2), log2f(l));
    if (a.stat) a.stat[row] = make_float2(M, 1.f / l);
}

// A cluster per segment (a.cluster CTAs of four warps, equal runs of its
// blocks). Row r is finished by CTA r % cluster, which has a place for every
// CTA's part of it. 122,880 keys x 24 heads (1.51 GB): 213 to 226 us, 6.7 to
// 7.1 TB/s, the measured copy rate; 6,144 listed keys x 24 heads 16 us with 11
// of them the bytes; 101 keys x 3 heads 3.6 us, of which 2 are the launch and
// the rest length -> page id -> keys -> join, one after another. A warp alone
// on its scheduler takes about 1,500 cycles per step of 32 keys (of single
// blocks, 16 keys, it took 1,000 each), whatever the depth of its ring and with
// half the products too: the four warps' copies and fragment loads are 128 KB
// a step through the SM's shared memory, 1,000 cycles. So few segments want
// many CTAs.
template <typename T, int NT, bool kWeigh> __global__ void __launch_bounds__(kWarps * 32) k_paged_attn_cluster(AttnArgs a) {
    constexpr int KV = Frag<NT>::kv;
    extern __shared__ __align__(128) unsigned char smem[];
    // [cluster][rows of this CTA]: a power of two times ceil(rows / it), 16 at most
    __shared__ __align__(16) float s_part[kRows][kD];
    __shared__ __align__(16) float4 s_pml[kRows];
    __shared__ float s_f[kRows];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, CS = a.cluster;
    const int lg = __ffs(CS) - 1;  // CS is a power of two
    const int rank = (int)(blockIdx.x & (CS - 1)), segment = (int)(blockIdx.x >> lg);
    grid_wait();
    if (CS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int bh = segment / a.rc;
    const Segment sg = segment_of(a, bh, segment % a.rc);
    const int len = paged_len(a.p, sg.b), nb = seg_blocks(a, a.idx ? bh : sg.b);
    const int per = (nb + CS * kWarps - 1) / (CS * kWarps);
    const int blk0 = min((rank * kWarps + wid) * per, nb), nblk = min(per, nb - blk0);
    float m_run[Frag<NT>::R], l_run[Frag<NT>::R], w_run[Frag<NT>::R], acc[Frag<NT>::A][4];
    attend_blocks<T, NT, kWeigh>(a, sg, len, blk0, nblk, ptx::smem_addr(smem) + wid * kStages * stage_bytes<KV>, m_run, l_run,
                                 w_run, acc);
    grid_go();
    T *out = static_cast<T *>(a.out);
    const float sl2 = log2_scale(a);
    if (CS == 1) {
        join_warps<NT>(
            smem, sg.rows, sl2, m_run, l_run, w_run, acc, true,
            [&](int row, float4 s) { store_row(a, sg.hq0 + row, s.x, s.y, sl2); },
            [&](int row, float4 o) {
                *reinterpret_cast<uint2 *>(out + (sg.hq0 + row) * kD + 4 * lane) = pack4<T>(o);
            });
        return;
    }
    const int own = (sg.rows + CS - 1) >> lg;  // rows a CTA finishes at most
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster runs
    const auto part = [&](int row) { return rank * own + (row >> lg); };
    const auto to = [&](int row) { return (uint32_t)(row & (CS - 1)); };
    join_warps<NT>(
        smem, sg.rows, sl2, m_run, l_run, w_run, acc, false,
        [&](int row, float4 s) { st_cluster4(ptx::cluster_addr(ptx::smem_addr(&s_pml[part(row)]), to(row)), s); },
        [&](int row, float4 o) {
            st_cluster4(ptx::cluster_addr(ptx::smem_addr(&s_part[part(row)][4 * lane]), to(row)), o);
        });
    ptx::cluster_sync();  // the parts are there
    if (tid < CS * own) {  // their weights, side by side
        const int at = tid % own, row = (at << lg) + rank;
        float M = -INFINITY, l = 0.f, w = 0.f;
        for (int c = 0; c < CS; ++c) M = fmaxf(M, s_pml[c * own + at].x);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
        for (int c = 0; c < CS; ++c) {
            const float4 s = s_pml[c * own + at];
            const float f = beside(s.x, ref, sl2);
            l += f * s.y;
            w += f * s.z;
        }
        s_f[tid] = w == 0.f ? 0.f : beside(s_pml[tid].x, ref, sl2) * own_weight<KV>(s_pml[tid].z) / w;
        if (tid < own && row < sg.rows) store_row(a, sg.hq0 + row, M, l, sl2);
    }
    __syncthreads();
    for (int at = 0, row = rank; row < sg.rows; ++at, row += CS) {
        float o = 0.f;
#pragma unroll 4
        for (int c = 0; c < CS; ++c) o += s_f[c * own + at] * s_part[c * own + at][tid];
        out[(sg.hq0 + row) * kD + tid] = from_f<T>(o);
    }
}

// Equal runs of all segments' blocks. A segment counts kLead blocks more than
// it has, in front of its own. 64 sequences of 37 to 16,000 keys x 8 heads
// (504 MB): 82 to 84 us with the join, 88 to 90% of the measured copy rate (99% at
// four times the bytes); of the rest 3.5 us are the start of a CTA (scan, length,
// page id, first keys) and 4 the join.
// Two CTAs per SM, as many as the grid has: unasked, the compiler took 168 registers and spills for three in the 8-bit walk (24
// heads of 122,880 keys 118 -> 127 us).
template <typename T, int NT, bool kWeigh> __global__ void __launch_bounds__(kWarps * 32, 2) k_paged_attn_runs(AttnArgs a) {
    constexpr int KV = Frag<NT>::kv, kFront = KV == 8 ? kLead8 : kLead;
    extern __shared__ __align__(128) unsigned char smem[];
    const Paged &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    grid_wait();
    const int N = a.idx ? p.B * p.Hkv : p.B;       // list entries
    const int mult = a.idx ? a.rc : p.Hkv * a.rc;  // segments per entry
    auto weight = [&](int n) {
        const int nb = seg_blocks(a, n);
        return nb > 0 ? nb + kFront : 0;
    };
    const Run run = find_run<kWarps>(
        N, [&](int n) -> long long { return (long long)weight(n) * mult; }, kCtas * kWarps, 1, kWarps);
    if (run.x0 >= run.x1) return;
    int n = min(run.n, N - 1), nb = weight(n);
    long long before = run.before;
    // the CTA's run lies in one segment: its warps' results are joined
    const int sub0 = clampi(div_small(run.x0 - before, max(nb, 1)), 0, mult - 1);
    const bool joined = run.x1 <= before + (long long)(sub0 + 1) * nb;
    long long x = min(run.x0 + wid * run.per, run.x1);
    const long long x_end = min(x + run.per, run.x1);
    T *out = static_cast<T *>(a.out);
    const float sl2 = log2_scale(a);
    while (joined || x < x_end) {  // a joined CTA's warp without blocks still brings its empty part
        if (!joined && x >= before + (long long)nb * mult) {  // also passes over entries without keys
            before += (long long)nb * mult;
            if (++n >= N) return;
            nb = weight(n);
            continue;
        }
        const int sub = joined ? sub0 : clampi(div_small(x - before, max(nb, 1)), 0, mult - 1);
        const long long seg0 = before + (long long)sub * nb;  // the segment's first block
        int off = (int)(x - seg0), take = (int)min((long long)(nb - off), x_end - x);
        const bool first = joined ? run.x0 == seg0 : off == 0;
        const bool last = joined ? run.x1 == seg0 + nb : off + take == nb;
        x += take;
        {   // the piece's own blocks: those behind the lead
            const int skip = clampi(kFront - off, 0, take);
            off += skip - kFront;
            take -= skip;
        }
        const int chunk = sub % a.rc, bh = a.idx ? n : n * p.Hkv + sub / a.rc;
        const Segment sg = segment_of(a, bh, chunk);
        const int len = paged_len(p, sg.b);
        float m_run[Frag<NT>::R], l_run[Frag<NT>::R], w_run[Frag<NT>::R], acc[Frag<NT>::A][4];
        attend_blocks<T, NT, kWeigh>(a, sg, len, off, take, ptx::smem_addr(smem) + wid * kStages * stage_bytes<KV>, m_run,
                                     l_run, w_run, acc);
        if (x >= x_end) grid_go();

        // A piece of the segment that begins it describes all of its pieces.
        const long long slot = 2LL * ((int)blockIdx.x * kWarps + (joined ? 0 : wid)) + (first ? 1 : 0);
        if (first && lane == 0 && (!joined || wid == 0)) {
            const long long s1 = seg0 + nb, cta = run.per * kWarps;
            const int w0 = (int)(seg0 / run.per), w_last = (int)((s1 - 1) / run.per);
            const int ca = (int)((seg0 + cta - 1) / cta);
            const int cb = (int)(s1 == run.total ? (s1 + cta - 1) / cta : s1 / cta);
            int4 d = make_int4(w0, w_last + 1 - w0, 0, w_last + 1 - w0);
            if (cb > ca) {
                d.y = ca * kWarps - w0;
                d.z = cb - ca;
                d.w = d.y + d.z + max(0, w_last + 1 - cb * kWarps);
            }
            a.seg[(long long)bh * a.rc + chunk] = d;
        }
        if (joined) {
            const bool whole = first && last;
            join_warps<NT>(
                smem, sg.rows, sl2, m_run, l_run, w_run, acc, whole,
                [&](int row, float4 s) {
                    if (whole)
                        store_row(a, sg.hq0 + row, s.x, s.y, sl2);
                    else
                        a.ml[slot * a.rows + row] = s;
                },
                [&](int row, float4 o) {
                    if (whole)
                        *reinterpret_cast<uint2 *>(out + (sg.hq0 + row) * kD + 4 * lane) = pack4<T>(o);
                    else
                        *reinterpret_cast<float4 *>(a.o + (slot * a.rows + row) * kD + 4 * lane) = o;
                });
            return;
        }
#pragma unroll
        for (int r = 0; r < Frag<NT>::R; ++r) {
            const int row = Frag<NT>::row(r);
            if (row >= sg.rows) continue;
            if (first && last) {
                const float inv = KV == 8 ? 1.f : w_run[r] == 0.f ? 0.f : 1.f / w_run[r];
                T *dst = out + (sg.hq0 + row) * kD;
                Frag<NT>::each(acc, r, [&](int d, float2 x) {
                    *reinterpret_cast<uint32_t *>(dst + d) = pack2<T>(x.x * inv, x.y * inv);
                });
                if (Frag<NT>::tells()) store_row(a, sg.hq0 + row, m_run[r], l_run[r], sl2);
            } else {
                float *dst = a.o + (slot * a.rows + row) * kD;
                Frag<NT>::each(acc, r, [&](int d, float2 x) { *reinterpret_cast<float2 *>(dst + d) = x; });
                if (Frag<NT>::tells()) a.ml[slot * a.rows + row] = make_float4(m_run[r], l_run[r], w_run[r], 0.f);
            }
        }
    }
}

// Writes the rows (sequence, query head) without keys and joins the pieces
// of the segments that crossed runs: W warps per row, R rows per CTA. The
// pieces' weights come first, all at once; then the warps take turns on the
// pieces, each with kJoinDeep loads in flight, and their sums are added in
// order (one head of 122,880 keys, 304 pieces: 20 us with its streaming; a
// running maximum over one piece after another took 48). Many rows have few
// pieces each, few rows many: kJoinFew rows and fewer get 16 warps each,
// kJoinMany and more one (8,192 rows: 43 -> 37 us with their streaming).
constexpr int kJoinDeep = 8, kJoinFew = 152, kJoinMany = 1024;
template <typename T, int KV, int W, int R> __global__ void __launch_bounds__(W * R * 32) k_paged_join(AttnArgs a) {
    static_assert(W == 1 || R == 1, "a row's warps meet at the CTA's barrier");
    __shared__ float s_ft[R][kCtas * kWarps], s_red[W], s_l[W], s_w[W];
    __shared__ __align__(16) float s_o[W][kD];
    const Paged &p = a.p;
    const int lane = threadIdx.x & 31, wid = R > 1 ? 0 : (int)threadIdx.x >> 5;  // warp of the row
    const int team = R > 1 ? (int)threadIdx.x >> 5 : 0, tid = wid * 32 + lane;
    const int row = blockIdx.x * R + team;
    grid_wait();
    grid_go();
    if (row >= p.B * p.Hq) return;
    const int b = row / p.Hq, hq = row % p.Hq, h = hq / p.G, in = hq % p.G;
    const int bh = b * p.Hkv + h;
    float *s_f = s_ft[team];
    T *out = static_cast<T *>(a.out) + (long long)row * kD;
    const int4 sg = a.seg[(long long)bh * a.rc + in / a.rows];  // not written for a segment without keys
    if (seg_keys(a, a.idx ? bh : b) == 0) {
        for (int d = tid; d < kD; d += W * 32) out[d] = from_f<T>(0.f);
        if (tid == 0) a.lse[row] = -INFINITY;
        return;
    }
    if (sg.w == 1) return;  // finished where it was computed
    const int r = in % a.rows, pieces = min(sg.w, kCtas * kWarps);
    // warps before the first joined CTA, joined CTAs (at their first warp's place), warps after
    auto place = [&](int i) {
        const int w = i < sg.y ? sg.x + i : (i < sg.y + sg.z ? sg.x + sg.y + (i - sg.y) * kWarps
                                                            : sg.x + i + sg.z * (kWarps - 1));
        return (2LL * clampi(w, 0, kCtas * kWarps - 1) + (i == 0 ? 1 : 0)) * a.rows + r;
    };
    const float sl2 = log2_scale(a);
    float M = -INFINITY;
    for (int i = tid; i < pieces; i += W * 32) {
        s_f[i] = a.ml[place(i)].x;
        M = fmaxf(M, s_f[i]);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (W > 1) {
        if (lane == 0) s_red[wid] = M;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, s_red[w]);
    }
    const float ref = M == -INFINITY ? 0.f : M;
    float l = 0.f, w = 0.f;
    for (int i = tid; i < pieces; i += W * 32) {  // the thread's own entries again
        const float e = beside(s_f[i], ref, sl2);
        const float4 s = a.ml[place(i)];
        s_f[i] = e * own_weight<KV>(s.z);
        l += e * s.y;
        w += e * s.z;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, off);
        w += __shfl_xor_sync(0xffffffffu, w, off);
    }
    if (W > 1) {
        if (lane == 0) s_l[wid] = l, s_w[wid] = w;
        __syncthreads();
    } else {
        __syncwarp();
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = wid; i0 < pieces; i0 += W * kJoinDeep) {
        float4 x[kJoinDeep];
#pragma unroll
        for (int e = 0; e < kJoinDeep; ++e)
            x[e] = i0 + e * W < pieces ? *reinterpret_cast<const float4 *>(a.o + place(i0 + e * W) * kD + 4 * lane)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int e = 0; e < kJoinDeep; ++e) {
            const float f = i0 + e * W < pieces ? s_f[i0 + e * W] : 0.f;
            o.x += f * x[e].x;
            o.y += f * x[e].y;
            o.z += f * x[e].z;
            o.w += f * x[e].w;
        }
    }
    if (W == 1) {
        const float inv = w == 0.f ? 0.f : 1.f / w;
        *reinterpret_cast<uint2 *>(out + 4 * lane) = pack4<T>(make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (lane == 0) store_row(a, row, M, l, sl2);
        return;
    }
    *reinterpret_cast<float4 *>(&s_o[wid][4 * lane]) = o;
    __syncthreads();
    if (tid >= kD) return;
    float val = 0.f;
    l = w = 0.f;
#pragma unroll
    for (int c = 0; c < W; ++c) {
        l += s_l[c];
        w += s_w[c];
        val += s_o[c][tid];
    }
    out[tid] = from_f<T>(w == 0.f ? 0.f : val / w);
    if (tid == 0) store_row(a, row, M, l, sl2);
}

// Whether clusters of 2 c CTAs take segments of up to `keys` keys better than
// clusters of c. The GPU has places for 152, 74, 36 and 14 clusters of 2, 4, 8
// and 16 CTAs; one more than that starts when another ends (15 segments of
// 16,000 keys in clusters of 8 / 16: 25.0 / 31.5 us, 14: 24.2 / 21.3), and a few
// less leave the SMs' loads more even (36 of 4,000, 4 / 8: 15.9 / 18.1). A
// cluster's barriers and join cost 1 to 2 us against 0.7 per 128 keys of a CTA:
// clusters of 1 / 2 / 4 took 4.1 / 4.5 / 4.4 for 200 keys x 14 heads, 5.7 / 5.4 /
// 4.4 for 400, 6.1 / 6.5 / - for 400 x 80, 12.0 / 11.1 / - for 1,000; of 4 / 8 / 16
// 5.5 / 4.8 / 5.7 for 1,000 x 14, 7.2 / 6.2 / 5.6 for 2,000.
inline bool grows(int c, long long segments, long long keys) {
    if (c == 1) return segments <= 72 ? keys > 320 : segments <= 152 && keys > 1024;
    if (c == 2) return segments <= 72;
    return c == 4 ? segments <= 32 && keys > 768 : segments <= 14 && keys > 1024;
}

// NT: the tiles of heads of an 8-bit cache's walk, 0: 16 bits.
template <typename T, int NT, bool kWeigh> vsa_status launch_attn(const AttnArgs &a, cudaStream_t s) {
    constexpr int KV = Frag<NT>::kv, smem = smem_bytes<KV>;
    if (a.cluster) {
        const auto kernel = k_paged_attn_cluster<T, NT, kWeigh>;
        cudaError_t e = ensure_smem_limit((const void *)kernel, smem);
        if (e == cudaSuccess && a.cluster > 8) e = ensure_wide_clusters((const void *)kernel);
        if (e != cudaSuccess) return status_from_cuda(e);
        prof_begin(KV == 8 ? "paged8_attn" : "paged_attn", s);
        e = launch_paged(kernel, dim3((unsigned)((long long)a.p.B * a.p.Hkv * a.rc * a.cluster)), kWarps * 32, smem,
                         a.cluster, a, s);
        prof_end(s);
        return status_from_cuda(e);
    }
    const auto kernel = k_paged_attn_runs<T, NT, kWeigh>;
    cudaError_t e = ensure_smem_limit((const void *)kernel, smem);
    if (e != cudaSuccess) return status_from_cuda(e);
    prof_begin(KV == 8 ? "paged8_attn" : "paged_attn", s);
    e = launch_paged(kernel, dim3(kCtas), kWarps * 32, smem, 1, a, s);
    prof_end(s);
    if (e != cudaSuccess) return status_from_cuda(e);
    prof_begin("paged_join", s);
    const unsigned out_rows = (unsigned)(a.p.B * a.p.Hq);
    e = out_rows <= kJoinFew   ? launch_paged(k_paged_join<T, KV, 16, 1>, dim3(out_rows), 512, 0, 1, a, s)
        : out_rows < kJoinMany ? launch_paged(k_paged_join<T, KV, 4, 1>, dim3(out_rows), 128, 0, 1, a, s)
                               : launch_paged(k_paged_join<T, KV, 1, 4>, dim3((out_rows + 3) / 4), 128, 0, 1, a, s);
    prof_end(s);
    return status_from_cuda(e);
}

// The checks and the choice of a kernel that all of the entry points share.
inline vsa_status attn_args(const AttnCall &c, bool eight, AttnArgs *args) {
    AttnArgs &a = *args;
    const vsa_status st = to_paged(c.desc, &a.p, true);
    if (st != VSA_OK) return st;
    if (eight && a.p.page_stride % 16 != 0) return VSA_ERR_SHAPE;
    if (!token_stride(c.q_stride, a.p.Hq, &a.qs)) return VSA_ERR_SHAPE;
    if (!c.q || !c.k || !c.v || !c.out || !c.lse || !c.idx != !c.cnt) return VSA_ERR_NULL;
    if (eight && (!c.ks || !c.vs)) return VSA_ERR_NULL;
    if (c.idx && c.cap < 1) return VSA_ERR_SHAPE;
    if (c.idx && (long long)c.cap * a.p.page > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    if (!aligned16(c.q) || !aligned16(c.k) || !aligned16(c.v) || !aligned16(c.out)) return VSA_ERR_LAYOUT;
    if (((uintptr_t)c.idx | (uintptr_t)c.cnt | (uintptr_t)c.lse | (uintptr_t)c.ks | (uintptr_t)c.vs) & 3u)
        return VSA_ERR_LAYOUT;
    const PagedWs ws = paged_ws(a.p);
    if (!c.ws || ((uintptr_t)c.ws & 255u) || c.ws_bytes < (c.weigh ? weigh_bytes(a.p) : ws.total)) return VSA_ERR_WORKSPACE;
    a.q = c.q;
    a.k = c.k;
    a.v = c.v;
    a.ks = c.ks;
    a.vs = c.vs;
    a.idx = c.idx;
    a.cnt = c.cnt;
    a.cap = c.cap;
    a.out = c.out;
    a.lse = c.lse;
    a.rows = rows_of(a.p.G);
    a.rc = (a.p.G + a.rows - 1) / a.rows;
    const long long most = c.idx ? std::min((long long)c.cap * a.p.page, (long long)a.p.max_len) : a.p.max_len;
    // One cluster per segment, its CTAs doubled while all of the clusters find a place at once and the keys are many
    // enough (grows()). Segments of one length (one sequence, or page lists) are then balanced by themselves; of
    // unknown lengths only while the longest stays short: the table's width stands for it, so that short sequences in a
    // wide table go to runs too (101 keys x 3 heads 3.2 us, in a table for 131,072 keys 7.2). Measured (us, clusters /
    // runs): 400 keys x 14 heads 4.4 / 8.2, x 400 19.5 / 21.8, x 1,600 61.6 / 60.9; 4,000 x 8 6.9 / 9.6, 64,000 x 24
    // 116 / 124, 64,000 x 1 34 / 13.6; 16 sequences of 1,000 to 9,000 keys x 2 heads 18.8 / 21.1, 64 of 37 to 16,000 x
    // 8 151 / 84.
    const long long segments = (long long)a.p.B * a.p.Hkv * a.rc;
    int cluster = 1;
    while (cluster < kMaxCluster && grows(cluster, segments, most)) cluster *= 2;
    // An 8-bit cache's runs keep more warps on each SM than a cluster's place on it leaves: 24 heads of 4,000, 16,000,
    // 122,880 keys 8.9 / 10.9, 25.2 / 19.7, 145 / 117.
    const bool even = !eight && (c.idx || a.p.B == 1);
    const bool few = most <= (long long)(eight ? kAlignedKeys8 : kAlignedKeys) * cluster && segments * cluster <= kFewCtas;
    a.cluster = few || (even && segments * cluster >= kAlignedCtas) ? cluster : 0;
    char *w = static_cast<char *>(c.ws);
    a.seg = reinterpret_cast<int4 *>(w + ws.seg);
    a.ml = reinterpret_cast<float4 *>(w + ws.ml);
    a.o = reinterpret_cast<float *>(w + ws.o);
    if (c.weigh) {
        a.stat = reinterpret_cast<float2 *>(w + ws.stat);
        a.bw = reinterpret_cast<float2 *>(w + ws.total);
        a.blocks = a.p.max_len / kBlk;
    }
    return VSA_OK;
}

}  // namespace
}  // namespace vsa
