// paged_rows.cuh -- what the appends to a 16-bit and to an 8-bit cache share:
// their arguments and checks, and which warp has which tokens. Internal.
//
// A unit is one page of one sequence that receives tokens. Units are found
// without a scan of the lengths: sequence b with tokens [cu[b], cu[b+1]) touches at most (cu[b+1] - cu[b]) / page + 2 pages, so
// numbering its units from cu[b] / page + 2 b leaves room for them, and a
// warp finds its b with a 32-way search of that ascending sequence.
#pragma once

#include <algorithm>

#include "paged.cuh"

namespace vsa {
namespace {

struct AppendArgs {
    Paged p;
    int T;
    const void *k, *v, *q;
    long long ks, vs, qs;       // elements between tokens
    void *q_out;
    const int *cu, *pos;
    const float *cos, *sin;
    int rows, rot, inter;       // table rows, rotated dims, interleaved pairs
    void *kc, *vc;
    float *mean;
    float *kscale, *vscale;     // 8 bits: scales [num_pages, Hkv, page / 16]
    long long units;
    int kv_chunks, chunks;  // chunks of key/value heads, and with the queries'
    int team;               // warps per unit
    int hc;                 // 8 bits: key/value heads per chunk
    int single;             // 8 bits: one token per sequence
};

constexpr int kGroup = 16;  // slots per warp, and tokens that share a scale

// First token of sequence b, clamped into [0, T].
__device__ __forceinline__ int cu_at(const AppendArgs &a, int b) { return clampi(a.cu[b], 0, a.T); }

// The sequence whose units hold unit u: the largest b with cu[b] / page +
// 2 b <= u. Whole warp, same u.
__device__ __forceinline__ int find_seq(const AppendArgs &a, long long u, int lane) {
    int lo = 0, n = a.p.B;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const int b = lo + lane * step;
        const bool le = lane * step < n && (cu_at(a, b) >> a.p.page_log2) + 2LL * b <= u;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int last = m ? 31 - __clz(m) : 0;
        const int end = lo + n;
        lo += last * step;
        n = min(step, end - lo);
    }
    return lo;
}

// cos / sin of the lane's 8 dims [8 i, 8 i + 8), by pair.
struct Angles {
    float c[8], s[8];  // half style: one per dim; interleaved: the first 4, one per pair
};
__device__ __forceinline__ void load4(float *dst, const float *src) {
    const float4 x = *reinterpret_cast<const float4 *>(src);
    dst[0] = x.x, dst[1] = x.y, dst[2] = x.z, dst[3] = x.w;
}
__device__ __forceinline__ void load_angles(const AppendArgs &a, int row, int i, Angles &w) {
    const int half = a.rot >> 1;
    const long long at = (long long)row * half;
    if (a.inter) {
        load4(w.c, a.cos + at + 4 * i);
        load4(w.s, a.sin + at + 4 * i);
    } else {
        const int d = 8 * i < half ? 8 * i : 8 * i - half;
        load4(w.c, a.cos + at + d);
        load4(w.c + 4, a.cos + at + d + 4);
        load4(w.s, a.sin + at + d);
        load4(w.s + 4, a.sin + at + d + 4);
    }
}

// Unit u: page `pg` of sequence b takes new tokens at slots [s0, s1); slot s
// holds token t_of + s. Empty (s0 == s1) where there are none.
struct Unit {
    int b, pg, s0, s1, t_of;
};
__device__ __forceinline__ Unit find_unit(const AppendArgs &a, long long u, int lane) {
    const Paged &p = a.p;
    Unit r{0, 0, 0, 0, 0};
    if (u >= a.units) return r;
    int t0, n;
    if (a.cu) {
        r.b = find_seq(a, u, lane);
        t0 = cu_at(a, r.b);
        n = max(cu_at(a, r.b + 1) - t0, 0);
    } else {
        r.b = (int)u;
        t0 = r.b;
        n = 1;
    }
    const long long len = p.lens[r.b], first = len - n;  // unclamped: positions outside are dropped
    const long long lo = max(first, 0LL), hi = min(len, (long long)p.max_len);
    const long long base = a.cu ? (t0 >> p.page_log2) + 2LL * r.b : u;
    const long long pl = (lo >> p.page_log2) + (u - base);
    const long long at = pl << p.page_log2;
    if (n > 0 && lo < hi && at < hi) {
        r.pg = (int)pl;
        r.s0 = (int)max(lo - at, 0LL);
        r.s1 = (int)min(hi - at, (long long)p.page);
        r.t_of = (int)(t0 + (at - first));
    }
    return r;
}

// Rotates the lane's 8 dims of a row held by 16 lanes. Each product and sum
// is rounded to fp32 by itself (no contraction), so the stored bits follow
// from the definition. All lanes of the warp take part.
template <typename T>
__device__ __forceinline__ uint4 rotate(const AppendArgs &a, uint4 x, const Angles &w, int i) {
    uint32_t r[4] = {x.x, x.y, x.z, x.w};
    if (a.inter) {
        if (8 * i < a.rot) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 e = unpack2<T>(r[j]);
                r[j] = pack2<T>(__fsub_rn(__fmul_rn(e.x, w.c[j]), __fmul_rn(e.y, w.s[j])),
                                __fadd_rn(__fmul_rn(e.y, w.c[j]), __fmul_rn(e.x, w.s[j])));
            }
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    }
    // the other element of each pair sits rot / 16 lanes away
    const int hop = a.rot >> 4;
    const bool on = 8 * i < a.rot, lower = i < hop;
    const int peer = (threadIdx.x & 16) | (on ? (lower ? i + hop : i - hop) : i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t o = __shfl_sync(0xffffffffu, r[j], peer);
        const float2 e = unpack2<T>(r[j]), f = unpack2<T>(o);
        const float sx = lower ? -w.s[2 * j] : w.s[2 * j], sy = lower ? -w.s[2 * j + 1] : w.s[2 * j + 1];
        // lower: x1 c - x2 s = x1 c + x2 (-s), the same bits; upper: x2 c + x1 s
        const uint32_t y = pack2<T>(__fadd_rn(__fmul_rn(e.x, w.c[2 * j]), __fmul_rn(f.x, sx)),
                                    __fadd_rn(__fmul_rn(e.y, w.c[2 * j + 1]), __fmul_rn(f.y, sy)));
        r[j] = on ? y : r[j];
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// rotate() of a whole head (128 dims) in one style: the same bits.
template <typename T, bool kInter> __device__ __forceinline__ uint4 rotate_all(uint4 x, const Angles &w, bool lower) {
    uint32_t r[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 e = unpack2<T>(r[j]);
        if constexpr (kInter) {
            r[j] = pack2<T>(__fsub_rn(__fmul_rn(e.x, w.c[j]), __fmul_rn(e.y, w.s[j])),
                            __fadd_rn(__fmul_rn(e.y, w.c[j]), __fmul_rn(e.x, w.s[j])));
        } else {
            const float2 f = unpack2<T>(__shfl_xor_sync(0xffffffffu, r[j], 8));
            const float sx = lower ? -w.s[2 * j] : w.s[2 * j], sy = lower ? -w.s[2 * j + 1] : w.s[2 * j + 1];
            r[j] = pack2<T>(__fadd_rn(__fmul_rn(e.x, w.c[2 * j]), __fmul_rn(f.x, sx)),
                            __fadd_rn(__fmul_rn(e.y, w.c[2 * j + 1]), __fmul_rn(f.y, sy)));
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// The rotated queries of a unit's tokens, heads h0 .. h0 + 2 HC - 1: a warp
// takes the 16-slot groups first_grp, first_grp + team, .. kStyle: 0 any
// rotation; all dims, interleaved (1) or not (2), at the tokens' positions.
template <typename T, int HC, int PB, int kStyle = 0>
__device__ __forceinline__ void append_queries(const AppendArgs &a, const Unit &of, int h0, int first_grp) {
    const Paged &p = a.p;
    const int lane = threadIdx.x & 31, half = lane >> 4, i = lane & 15;
    const int s0 = of.s0, s1 = of.s1, pg = of.pg, t_of = of.t_of, hn = min(2 * HC, p.Hq - h0);
    const T *q = static_cast<const T *>(a.q);
    T *qo = static_cast<T *>(a.q_out);
    for (int st = first_grp * kGroup; st < s1; st += 2 * PB) {
        if (st % kGroup == 0 && st != first_grp * kGroup) st += (a.team - 1) * kGroup;  // the warp's next group
        if (st >= s1 || st + 2 * PB <= s0) continue;
        uint4 x[PB][2 * HC];
        Angles w[PB];
#pragma unroll
        for (int c = 0; c < PB; ++c) {
            const int s = st + 2 * c + half;
            const bool fresh = s >= s0 && s < s1;
            const long long tok = fresh ? t_of + s : 0;
#pragma unroll
            for (int h = 0; h < 2 * HC; ++h)
                x[c][h] = fresh && h < hn
                              ? *reinterpret_cast<const uint4 *>(q + tok * a.qs + (h0 + h) * kD + 8 * i)
                              : make_uint4(0, 0, 0, 0);
            if constexpr (kStyle != 0) {
                const int row = min((pg << p.page_log2) + s, a.rows - 1);
                const long long at = (long long)row * 64 + (kStyle == 1 ? 4 * i : 8 * (i & 7));
                load4(w[c].c, a.cos + at);
                load4(w[c].s, a.sin + at);
                if constexpr (kStyle == 2) {
                    load4(w[c].c + 4, a.cos + at + 4);
                    load4(w[c].s + 4, a.sin + at + 4);
                }
            } else if (fresh && 8 * i < a.rot) {
                const int row = a.pos ? a.pos[tok] : (pg << p.page_log2) + s;
                load_angles(a, clampi(row, 0, a.rows - 1), i, w[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < PB; ++c) {
            const int s = st + 2 * c + half;
            const bool fresh = s >= s0 && s < s1;
            const long long tok = fresh ? t_of + s : 0;
#pragma unroll
            for (int h = 0; h < 2 * HC; ++h) {
                if constexpr (kStyle != 0)
                    x[c][h] = rotate_all<T, kStyle == 1>(x[c][h], w[c], i < 8);
                else if (a.rot)
                    x[c][h] = rotate<T>(a, x[c][h], w[c], i);
                if (fresh && h < hn)
                    *reinterpret_cast<uint4 *>(qo + (tok * p.Hq + h0 + h) * kD + 8 * i) = x[c][h];
            }
        }
    }
}

// Warps per unit: as many as a sequence's tokens fill groups on average (idle
// warps hold registers), and up to four for the earlier keys of a page that
// fills up.
inline int team_of(const AppendArgs &a) {
    const int groups = a.p.page / kGroup;
    int team = std::min(groups, 4);
    while (team < groups && (long long)a.T > (long long)team * kGroup * a.p.B) team *= 2;
    return team;
}

// Host: the checks of both appends, and their arguments. T == 0: nothing to do.
inline vsa_status append_args(const vsa_paged_desc *desc, int T, const void *k, int64_t k_stride, const void *v,
                              int64_t v_stride, const void *q, int64_t q_stride, void *q_out, const int32_t *cu_seqlens,
                              const int32_t *positions, const float *cos, const float *sin, int table_rows, int rot_dim,
                              int interleaved, void *k_cache, void *v_cache, float *k_mean, AppendArgs *args) {
    AppendArgs &a = *args;
    const vsa_status st = to_paged(desc, &a.p, true);
    if (st != VSA_OK) return st;
    if (T < 0 || (!cu_seqlens && T != a.p.B)) return VSA_ERR_SHAPE;
    if (!token_stride(k_stride, a.p.Hkv, &a.ks) || !token_stride(v_stride, a.p.Hkv, &a.vs) ||
        !token_stride(q_stride, a.p.Hq, &a.qs))
        return VSA_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim > kD || rot_dim % 16 != 0) return VSA_ERR_UNSUPPORTED;
    if (rot_dim > 0 && (!cos || !sin)) return VSA_ERR_NULL;
    if (rot_dim > 0 && table_rows < 1) return VSA_ERR_SHAPE;
    if (!q != !q_out || !k_cache || !v_cache) return VSA_ERR_NULL;
    if (T == 0) return VSA_OK;
    if (!k || !v) return VSA_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned16(k_mean))
        return VSA_ERR_LAYOUT;
    if (rot_dim > 0 && (!aligned16(cos) || !aligned16(sin))) return VSA_ERR_LAYOUT;
    if ((uintptr_t)cu_seqlens & 3u || (uintptr_t)positions & 3u) return VSA_ERR_LAYOUT;
    a.T = T;
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.cu = cu_seqlens;
    a.pos = positions;
    a.cos = cos;
    a.sin = sin;
    a.rows = table_rows;
    a.rot = rot_dim;
    a.inter = interleaved != 0;
    a.kc = k_cache;
    a.vc = v_cache;
    a.mean = k_mean;
    a.units = cu_seqlens ? (long long)T / a.p.page + 2LL * a.p.B : a.p.B;
    if (a.units * (a.p.Hkv + a.p.Hq) > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;  // more CTAs than a grid holds
    return VSA_OK;
}

}  // namespace
}  // namespace vsa
