// paged_attn.cu -- attention of one token per sequence over a paged
// key/value cache (vsa_paged_attn), all pages or the listed ones.
//
//   O = sum_u P_u v_u / sum_u P_u,  P_u = exp(scale q.k_u - max)
//
// A segment is one (sequence, key/value head, chunk of up to 16 query heads
// of its group: one tile of the tensor instructions; a wider group's chunks
// read the same keys, from L2 but for the first); its keys, in the order of the pages attended, are
// cut into blocks of 16. The blocks of all segments, end to end, are dealt
// to the grid's warps in equal contiguous runs, whatever the lengths of the
// batch: a CTA finds its run with one scan of the lengths, and each warp
// walks the segments of its own part of it. A segment inside one warp's run
// is finished there. Where a CTA's whole run lies in one segment its warps'
// results are joined in shared memory first; the remaining pieces of
// segments that cross runs go to the workspace (at most two per warp) and
// k_paged_join adds them in ascending order. When the table or the page
// lists allow only short segments (up to kAlignedKeys keys per CTA) each
// segment gets a CTA, or a cluster of CTAs that join through distributed
// shared memory, and one launch does it all.
//
// A warp takes its blocks through its own ring of asynchronous copies (16 K
// rows and 16 V rows of 256 bytes per stage, swizzled so that ldmatrix reads
// hit distinct banks; rows past a page's valid slots are filled with zeros,
// so whatever the cache holds there cannot reach the sums) and keeps its own
// running maximum, sum and output in registers: no warp waits for another
// while it streams. The products run on m16n8k16 tensor instructions with
// the group's query heads as rows. At one query token per sequence the
// kernel reads 512 bytes per 256 G multiply-adds, far to the memory side of
// the tensor cores' balance, so the instruction's rate does not bound it;
// the memory pipe does, and the loads in flight on it.
#include <algorithm>

#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace vsa {
namespace {

constexpr int kBlk = 16;        // keys per warp step
constexpr int kRows = 16;       // query heads per segment at most
constexpr int kLead = 4;        // blocks a segment counts for beyond its own (its start-up time)
constexpr int kMinBlocks = 4;   // fewest blocks a warp's run has when there is little work
constexpr int kAlignedKeys = 2048;  // keys per CTA up to which a segment is one CTA's or one cluster's
constexpr int kAlignedCtas = 96;    // CTAs that nearly fill the memory pipe
constexpr int kMaxCluster = 8;
constexpr int kWarps = 4;
constexpr int kStages = 3;      // ring stages per warp
constexpr int kCtas = 304;      // two per SM on 152 SMs
constexpr int kStageBytes = 2 * kBlk * 256;
constexpr int kPitch = 136;     // floats per row of the warps' outputs in shared memory
constexpr int kSmem = kWarps * kStages * kStageBytes;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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
    int aligned;           // CTAs per segment, one cluster; 0: equal runs of all segments' blocks
    int lead;              // kLead, 0 when aligned
    int4 *seg;             // [segments] its pieces: first warp, warps before / CTAs joined / pieces in all
    float2 *ml;            // [2 * kCtas * kWarps, rows]
    float *o;              // [2 * kCtas * kWarps, rows, 128]
};

// Keys of segment list entry n ((b) without page lists, (b, h) with): the
// positions it walks, valid or not.
__device__ __forceinline__ int seg_keys(const AttnArgs &a, int n) {
    if (!a.idx) return paged_len(a.p, n);
    return clampi(__ldg(a.cnt + n), 0, a.cap) * a.p.page;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool fill) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
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

// Blocks of a segment, its lead in front of its own counted in.
__device__ __forceinline__ int seg_blocks(const AttnArgs &a, int n) {
    const int nb = (seg_keys(a, n) + kBlk - 1) / kBlk;
    return nb > 0 ? nb + a.lead : 0;
}

template <typename T> __global__ void __launch_bounds__(kWarps * 32) k_paged_attn(AttnArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    __shared__ float2 s_cta[kRows];  // the CTA's own maximum and sum, for its cluster
    const Paged &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, t = lane & 3;
    grid_wait();
    grid_go();
    const int N = a.idx ? p.B * p.Hkv : p.B;             // list entries
    const int mult = a.idx ? a.rc : p.Hkv * a.rc;        // segments per entry
    const T *K = static_cast<const T *>(a.k), *V = static_cast<const T *>(a.v), *Q = static_cast<const T *>(a.q);
    const uint32_t ring = ptx::smem_addr(smem) + wid * kStages * kStageBytes;
    const float sl2 = p.scale * kLog2e;

    Run run;
    const int segment = a.aligned ? (int)(blockIdx.x / a.aligned) : 0;
    if (a.aligned) {
        run.n = segment / mult;
        const int nb = seg_blocks(a, run.n), at = (int)(blockIdx.x % a.aligned) * kWarps;
        run.per = (nb + a.aligned * kWarps - 1) / (a.aligned * kWarps);
        run.before = 0;
        run.x0 = (long long)(segment % mult) * nb + min((long long)at * run.per, (long long)nb);
        run.x1 = (long long)(segment % mult) * nb + min((long long)(at + kWarps) * run.per, (long long)nb);
        run.total = 0;
    } else {
        run = find_run<kWarps>(
            N, [&](int n) -> long long { return (long long)seg_blocks(a, n) * mult; }, kCtas * kWarps, kMinBlocks,
            kWarps);
        if (run.x0 >= run.x1) return;
    }
    // the CTA's run lies in one segment: its warps' results are joined
    bool joined = a.aligned;
    if (!a.aligned) {
        const int nb = seg_blocks(a, run.n);
        joined = (run.x0 - run.before) / nb == (run.x1 - 1 - run.before) / nb && run.x1 <= run.before + (long long)nb * mult;
    }
    long long x = min(run.x0 + wid * run.per, run.x1);
    const long long x_end = min(x + run.per, run.x1);
    int n = run.n;
    long long before = run.before;
    bool more = joined || x < x_end;  // a joined CTA's warp without blocks still brings its empty part
    while (more) {
        int nb = n < N ? seg_blocks(a, n) : 0;
        if (!joined && x >= before + (long long)nb * mult) {  // also passes over entries without keys
            before += (long long)nb * mult;
            if (++n >= N) break;
            continue;
        }
        long long seg0;   // first block of the segment
        int sub, off, take;
        if (joined) {     // the segment is the run's, also for a warp without blocks
            sub = a.aligned ? segment % mult : (int)((run.x0 - before) / nb);
            seg0 = before + (long long)sub * nb;
            off = (int)(x - seg0);
            take = (int)(x_end - x);
        } else {
            sub = (int)((x - before) / nb);
            seg0 = before + (long long)sub * nb;
            off = (int)(x - seg0);
            take = (int)min((long long)(nb - off), x_end - x);
        }
        const bool first = joined ? run.x0 == seg0 : off == 0;
        const bool last = joined ? run.x1 == seg0 + nb : off + take == nb;
        x += take;
        {   // the piece's own blocks: those behind the lead
            const int skip = clampi(a.lead - off, 0, take);
            off += skip - a.lead;
            take -= skip;
        }
        const int r = sub % a.rc, bh = a.idx ? n : n * p.Hkv + sub / a.rc;
        const int b = bh / p.Hkv, h = bh % p.Hkv;
        const int rows = min(a.rows, p.G - r * a.rows);
        const int len = paged_len(p, b);
        const int key0 = off * kBlk;
        const long long hoff = (long long)h * p.head_stride;

        // Q as A fragments: row g (and g + 8) of each 16-row tile, 8 k-steps
        uint32_t qa[8][4];
        {
            const T *qb = Q + (long long)b * a.qs + ((long long)h * p.G + r * a.rows) * kD;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = g + 8 * e;
                const uint32_t *src = reinterpret_cast<const uint32_t *>(qb + (long long)row * kD);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    qa[j][e] = row < rows ? __ldg(src + 8 * j + t) : 0u;
                    qa[j][2 + e] = row < rows ? __ldg(src + 8 * j + 4 + t) : 0u;
                }
            }
        }

        // Window of up to 32 blocks, one per lane: the page (or -1), the
        // slot in it and the valid slots of the block.
        int w_id = -1, w_slot = 0, w_valid = 0, w_base = -32;
        auto window = [&](int i0) {
            w_base = i0;
            w_id = -1;
            w_valid = 0;
            if (i0 + lane < take) {
                const int pos = key0 + (i0 + lane) * kBlk;
                int j = pos >> p.page_log2;
                w_slot = pos & (p.page - 1);
                if (a.idx) j = __ldg(a.idx + (long long)bh * a.cap + j);
                w_id = paged_id(p, b, j);
                if (w_id >= 0) w_valid = clampi(len - (j << p.page_log2) - w_slot, 0, kBlk);
            }
        };
        int valid[kStages];
        auto issue = [&](int i, int stage) {  // block i of this piece into a stage
            if (i >= w_base + 32) window(i);
            const int id = __shfl_sync(0xffffffffu, w_id, i - w_base);
            const int slot = __shfl_sync(0xffffffffu, w_slot, i - w_base);
            const int ok = __shfl_sync(0xffffffffu, w_valid, i - w_base);
            const long long at = (long long)max(id, 0) * p.page_stride + slot * p.tok_stride + hoff;
            const int c = lane & 15;
            const uint32_t dst = ring + stage * kStageBytes;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = 2 * e + (lane >> 4);
                const bool live = row < ok;
                const long long src = live ? at + row * p.tok_stride + 8 * c : 0;
                const uint32_t d = dst + row * 256 + ((c ^ (row & 7)) << 4);
                cp16(d, K + src, live);
                cp16(d + kBlk * 256, V + src, live);
            }
            return ok;
        };
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            valid[s] = 0;
            if (s < take) valid[s] = issue(s, s);
            cp_commit();
        }
        valid[kStages - 1] = 0;

        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f}, acc[16][4];  // rows g and g + 8
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
        for (int i0 = 0; i0 < take; i0 += kStages) {
#pragma unroll
            for (int s = 0; s < kStages; ++s) {
                const int i = i0 + s;
                if (i >= take) break;
                cp_wait<kStages - 2>();
                __syncwarp();  // every lane's copies of this block have landed, and the stage ahead is free
                const uint32_t st = ring + s * kStageBytes;
                // All K fragments before the products that use them: the loads' latency is paid once a block.
                uint32_t kb[8][4];
                {
                    const int row = (lane & 7) + ((lane >> 4) << 3), c0 = (lane >> 3) & 1;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ldsm4(kb[j], st + row * 256 + (((2 * j + c0) ^ (row & 7)) << 4));
                }
                if (i + kStages - 1 < take)
                    valid[(s + kStages - 1) % kStages] = issue(i + kStages - 1, (s + kStages - 1) % kStages);
                cp_commit();
                float sc[2][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[0][e] = sc[1][e] = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    mma16816<T>(sc[0], qa[j], kb[j][0], kb[j][1]);
                    mma16816<T>(sc[1], qa[j], kb[j][2], kb[j][3]);
                }
                // half of V's fragments, to arrive while the softmax runs
                const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8, vc0 = lane >> 4;
                auto ld_v = [&](uint32_t (&r)[4], int j) {
                    ldsm4t(r, st + kBlk * 256 + vrow * 256 + (((2 * j + vc0) ^ (vrow & 7)) << 4));
                };
                uint32_t vb[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) ld_v(vb[j], j);
                const int ok = valid[s];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = 8 * u + 2 * t + (e & 1);
                        sc[u][e] = key < ok ? sc[u][e] * sl2 : -INFINITY;
                    }
                float corr[2];
                bool moved = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(fmaxf(sc[0][2 * e], sc[0][2 * e + 1]), fmaxf(sc[1][2 * e], sc[1][2 * e + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float mn = fmaxf(m_run[e], mx);
                    const float ref = mn == -INFINITY ? 0.f : mn;  // a row without keys so far
                    corr[e] = ptx::ex2(m_run[e] - ref);
                    moved = moved || mn != m_run[e];
                    m_run[e] = mn;
                    float sum = 0.f;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float pr = ptx::ex2(sc[u][2 * e + c] - ref);
                            sc[u][2 * e + c] = pr;
                            sum += pr;
                        }
                    l_run[e] = l_run[e] * corr[e] + sum;  // this lane's keys; quads are joined at the end
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        acc[j][0] *= corr[0];
                        acc[j][1] *= corr[0];
                        acc[j][2] *= corr[1];
                        acc[j][3] *= corr[1];
                    }
                }
                // P <= 1 is rounded to the cache's 16-bit type for the product with V (the sum l keeps the
                // unrounded values): half a step of the output's own type
                const uint32_t pa[4] = {pack2<T>(sc[0][0], sc[0][1]), pack2<T>(sc[0][2], sc[0][3]),
                                        pack2<T>(sc[1][0], sc[1][1]), pack2<T>(sc[1][2], sc[1][3])};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    mma16816<T>(acc[2 * j], pa, vb[j & 3][0], vb[j & 3][1]);
                    mma16816<T>(acc[2 * j + 1], pa, vb[j & 3][2], vb[j & 3][3]);
                    if (j < 4) ld_v(vb[j], j + 4);
                }
            }
        }
        cp_wait<0>();
        __syncwarp();  // the warp's ring is free
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 1);
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 2);
        }
        const long long hq0 = (long long)b * p.Hq + h * p.G + r * a.rows;  // first output row of the segment

        // A piece of the segment that begins it describes all of its pieces.
        const int gw = (int)blockIdx.x * kWarps + (joined ? 0 : wid);
        const long long slot = 2LL * gw + (first ? 1 : 0);
        if (!a.aligned && first && lane == 0 && (!joined || wid == 0)) {
            const long long s1 = seg0 + nb, cta = run.per * kWarps;
            const int w_last = (int)((s1 - 1) / run.per);
            const int ca = (int)((seg0 + cta - 1) / cta);
            const int cb = (int)(s1 == run.total ? (s1 + cta - 1) / cta : s1 / cta);
            const int w0 = (int)(seg0 / run.per);
            int4 d = make_int4(w0, w_last + 1 - w0, 0, w_last + 1 - w0);
            if (cb > ca) {
                d.y = ca * kWarps - w0;
                d.z = cb - ca;
                d.w = d.y + d.z + max(0, w_last + 1 - cb * kWarps);
            }
            a.seg[(long long)bh * a.rc + r] = d;
        }

        if (joined) {  // the warps' outputs in shared memory, one thread per dim
            float *so = reinterpret_cast<float *>(smem + wid * kStages * kStageBytes);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = g + 8 * e;
                if (t == 0) {
                    s_m[wid][row] = m_run[e];
                    s_l[wid][row] = l_run[e];
                }
                if (row < rows)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        *reinterpret_cast<float2 *>(so + row * kPitch + 8 * j + 2 * t) =
                            make_float2(acc[j][2 * e], acc[j][2 * e + 1]);
            }
            __syncthreads();
            for (int row = 0; row < rows; ++row) {
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][row]);
                const float ref = M == -INFINITY ? 0.f : M;
                float l = 0.f, o = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = ptx::ex2(s_m[w][row] - ref);
                    l += f * s_l[w][row];
                    o += f * reinterpret_cast<const float *>(smem + w * kStages * kStageBytes)[row * kPitch + tid];
                }
                if (a.aligned > 1) {  // in place: this thread alone reads and writes the element
                    reinterpret_cast<float *>(smem)[row * kPitch + tid] = o;
                    if (tid == 0) s_cta[row] = make_float2(M, l);
                } else if (a.aligned || (first && last)) {
                    static_cast<T *>(a.out)[(hq0 + row) * kD + tid] = from_f<T>(l == 0.f ? 0.f : o / l);
                    if (tid == 0) a.lse[hq0 + row] = l == 0.f ? -INFINITY : kLn2 * (M + log2f(l));
                } else {
                    a.o[(slot * a.rows + row) * kD + tid] = o;
                    if (tid == 0) a.ml[slot * a.rows + row] = make_float2(M, l);
                }
            }
            if (a.aligned > 1) {  // the cluster's CTAs, each for its share of the rows
                ptx::cluster_sync();
                const uint32_t at_o = ptx::smem_addr(smem) + tid * 4, at_ml = ptx::smem_addr(s_cta);
                for (int row = (int)ptx::cluster_rank(); row < rows; row += a.aligned) {
                    float2 ml[kMaxCluster];
                    float o[kMaxCluster], M = -INFINITY, l = 0.f, sum = 0.f;
#pragma unroll
                    for (int c = 0; c < kMaxCluster; ++c) {
                        ml[c] = make_float2(-INFINITY, 0.f);
                        o[c] = 0.f;
                        if (c < a.aligned) {
                            ml[c] = ld_cluster2(ptx::cluster_addr(at_ml + row * 8, c));
                            o[c] = ld_cluster(ptx::cluster_addr(at_o + row * kPitch * 4, c));
                        }
                    }
#pragma unroll
                    for (int c = 0; c < kMaxCluster; ++c) M = fmaxf(M, ml[c].x);
                    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
                    for (int c = 0; c < kMaxCluster; ++c) {
                        const float f = ptx::ex2(ml[c].x - ref);
                        l += f * ml[c].y;
                        sum += f * o[c];
                    }
                    static_cast<T *>(a.out)[(hq0 + row) * kD + tid] = from_f<T>(l == 0.f ? 0.f : sum / l);
                    if (tid == 0) a.lse[hq0 + row] = l == 0.f ? -INFINITY : kLn2 * (M + log2f(l));
                }
                ptx::cluster_sync();  // no CTA leaves while another reads its part
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = g + 8 * e;
            if (row >= rows) continue;
            const float l = l_run[e];
            if (first && last) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + (hq0 + row) * kD);
#pragma unroll
                for (int j = 0; j < 16; ++j) dst[4 * j + t] = pack2<T>(acc[j][2 * e] * inv, acc[j][2 * e + 1] * inv);
                if (t == 0) a.lse[hq0 + row] = l == 0.f ? -INFINITY : kLn2 * (m_run[e] + log2f(l));
            } else {
                float *dst = a.o + (slot * a.rows + row) * kD;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    *reinterpret_cast<float2 *>(dst + 8 * j + 2 * t) = make_float2(acc[j][2 * e], acc[j][2 * e + 1]);
                if (t == 0) a.ml[slot * a.rows + row] = make_float2(m_run[e], l);
            }
        }
        more = x < x_end;
    }
}

// Writes the rows (sequence, query head) without keys and joins the pieces
// of the segments that crossed runs: W warps per row, R rows per CTA. The
// pieces' weights come first, all at once; then the warps take turns on the
// pieces, each with kJoinDeep loads in flight, and their sums are added in
// order. Many rows have few pieces each, few rows many: kJoinFew rows and
// fewer get 16 warps each, kJoinMany and more one.
constexpr int kJoinDeep = 8, kJoinFew = 152, kJoinMany = 1024;
template <typename T, int W, int R> __global__ void __launch_bounds__(W * R * 32) k_paged_join(AttnArgs a) {
    static_assert(W == 1 || R == 1, "a row's warps meet at the CTA's barrier");
    __shared__ float s_wt[R][kCtas * kWarps], s_red[W], s_sum[W];
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
    float *s_w = s_wt[team];
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
        return (2LL * w + (i == 0 ? 1 : 0)) * a.rows + r;
    };
    float M = -INFINITY;
    for (int i = tid; i < pieces; i += W * 32) {
        s_w[i] = a.ml[place(i)].x;
        M = fmaxf(M, s_w[i]);
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
    float l = 0.f;
    for (int i = tid; i < pieces; i += W * 32) {  // the thread's own entries again
        const float e = ptx::ex2(s_w[i] - ref);
        s_w[i] = e;
        l += e * a.ml[place(i)].y;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (W > 1) {
        if (lane == 0) s_sum[wid] = l;
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
            const float f = i0 + e * W < pieces ? s_w[i0 + e * W] : 0.f;
            o.x += f * x[e].x;
            o.y += f * x[e].y;
            o.z += f * x[e].z;
            o.w += f * x[e].w;
        }
    }
    if (W == 1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<uint2 *>(out + 4 * lane) = make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
        if (lane == 0) a.lse[row] = l == 0.f ? -INFINITY : kLn2 * (M + log2f(l));
        return;
    }
    *reinterpret_cast<float4 *>(&s_o[wid][4 * lane]) = o;
    __syncthreads();
    if (tid >= kD) return;
    float sum = 0.f, val = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        sum += s_sum[w];
        val += s_o[w][tid];
    }
    out[tid] = from_f<T>(sum == 0.f ? 0.f : val / sum);
    if (tid == 0) a.lse[row] = sum == 0.f ? -INFINITY : kLn2 * (M + log2f(sum));
}

// Rows per chunk of a group of G query heads: equal chunks of up to 16.
int rows_of(int G) {
    const int chunks = (G + kRows - 1) / kRows;
    return (G + chunks - 1) / chunks;
}

template <typename T> vsa_status launch_attn(const AttnArgs &a, cudaStream_t s) {
    const unsigned grid = a.aligned ? (unsigned)((long long)a.p.B * a.p.Hkv * a.rc * a.aligned) : kCtas;
    const unsigned cluster = a.aligned > 1 ? a.aligned : 1;
    cudaError_t e = ensure_smem_limit((const void *)k_paged_attn<T>, kSmem);
    if (e != cudaSuccess) return status_from_cuda(e);
    prof_begin("paged_attn", s);
    e = launch_paged(k_paged_attn<T>, grid, kWarps * 32, kSmem, cluster, a, s);
    prof_end(s);
    if (e != cudaSuccess || a.aligned) return status_from_cuda(e);
    prof_begin("paged_join", s);
    const unsigned out_rows = (unsigned)(a.p.B * a.p.Hq);
    e = out_rows <= kJoinFew    ? launch_paged(k_paged_join<T, 16, 1>, dim3(out_rows), 512, 0, 1, a, s)
        : out_rows < kJoinMany ? launch_paged(k_paged_join<T, 4, 1>, dim3(out_rows), 128, 0, 1, a, s)
                               : launch_paged(k_paged_join<T, 1, 4>, dim3((out_rows + 3) / 4), 128, 0, 1, a, s);
    prof_end(s);
    return status_from_cuda(e);
}

}  // namespace

PagedWs paged_ws(const Paged &p) {
    PagedWs w{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) & ~size_t(255);
        return o;
    };
    const size_t rows = rows_of(p.G), rc = (p.G + rows - 1) / rows;
    w.keys = take(sizeof(uint32_t) * p.B * (size_t)p.Hkv * p.max_pages);
    w.seg = take(sizeof(int4) * p.B * (size_t)p.Hkv * rc);
    w.ml = take(sizeof(float2) * 2 * kCtas * kWarps * rows);
    w.o = take(sizeof(float) * 2 * kCtas * kWarps * rows * kD);
    w.total = at;
    return w;
}

}  // namespace vsa

extern "C" size_t vsa_paged_workspace_size(const vsa_paged_desc *desc) {
    vsa::Paged p;
    if (vsa::to_paged(desc, &p, false) != VSA_OK) return 0;
    return vsa::paged_ws(p).total;
}

extern "C" vsa_status vsa_paged_attn(const vsa_paged_desc *desc, const void *q, int64_t q_stride,
                                     const void *k_cache, const void *v_cache, const int32_t *page_idx,
                                     const int32_t *page_cnt, int idx_cap, void *out, float *lse, void *workspace,
                                     size_t workspace_bytes, vsa_stream_t stream) {
    using namespace vsa;
    AttnArgs a{};
    const vsa_status st = to_paged(desc, &a.p, true);
    if (st != VSA_OK) return st;
    if (!token_stride(q_stride, a.p.Hq, &a.qs)) return VSA_ERR_SHAPE;
    if (!q || !k_cache || !v_cache || !out || !lse || !page_idx != !page_cnt) return VSA_ERR_NULL;
    if (page_idx && idx_cap < 1) return VSA_ERR_SHAPE;
    if (page_idx && (long long)idx_cap * a.p.page > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return VSA_ERR_LAYOUT;
    if (((uintptr_t)page_idx | (uintptr_t)page_cnt | (uintptr_t)lse) & 3u) return VSA_ERR_LAYOUT;
    const PagedWs ws = paged_ws(a.p);
    if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < ws.total) return VSA_ERR_WORKSPACE;
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.idx = page_idx;
    a.cnt = page_cnt;
    a.cap = idx_cap;
    a.out = out;
    a.lse = lse;
    a.rows = rows_of(a.p.G);
    a.rc = (a.p.G + a.rows - 1) / a.rows;
    const long long most = page_idx ? std::min((long long)idx_cap * a.p.page, (long long)a.p.max_len) : a.p.max_len;
    // One cluster per segment, the smallest that gives every SM a CTA. Segments of one length (one sequence, or
    // page lists) are then balanced by themselves; of unknown lengths only while the longest stays short.
    const long long segments = (long long)a.p.B * a.p.Hkv * a.rc;
    int cluster = 1;
    while (cluster < kMaxCluster && segments * cluster < 152) cluster *= 2;
    const bool even = page_idx || a.p.B == 1;
    const bool few = most <= (long long)kAlignedKeys * cluster && segments * cluster <= kCtas;
    a.aligned = few || (even && segments * cluster >= kAlignedCtas) ? cluster : 0;
    a.lead = a.aligned ? 0 : kLead;
    char *w = static_cast<char *>(workspace);
    a.seg = reinterpret_cast<int4 *>(w + ws.seg);
    a.ml = reinterpret_cast<float2 *>(w + ws.ml);
    a.o = reinterpret_cast<float *>(w + ws.o);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return a.p.dtype == T_BF16 ? launch_attn<__nv_bfloat16>(a, s) : launch_attn<__half>(a, s);
}
