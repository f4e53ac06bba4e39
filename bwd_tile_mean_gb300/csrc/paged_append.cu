// paged_append.cu -- new tokens' keys and values into the paged cache, keys
// and queries rotated by their positions on the way, and the mean key of
// every page that fills up (vsa_paged_append).
//
// Work: a unit is one page of one sequence that receives tokens; a warp has
// a 16-slot group of a unit (or some, in turns) and a chunk of rows per token: HC keys and
// values, or 2 HC queries. Half a warp holds one token row (16 bytes = 8
// dims per lane), the two halves the even and the odd slots; PB pairs of
// slots are loaded together. The rotation's angles are loaded once per token
// and chunk. Every key that a lane stores is also added, as stored, to the
// lane's running sums; in a page that fills up the slots written by earlier
// calls are read back from the cache in the same order, and the groups' sums
// are joined through shared memory.
//
// Units are found without a scan of the lengths: sequence b with tokens
// [cu[b], cu[b+1]) touches at most (cu[b+1] - cu[b]) / page + 2 pages, so
// numbering its units from cu[b] / page + 2 b leaves room for them, and a
// warp finds its b with a 32-way search of that ascending sequence.
//
// Bound by HBM for long prompts: 30,000 tokens of 24 heads (1.16 GB) take
// 191 us = 6.1 TB/s, 90% of the measured copy rate (97% without a rotation:
// the rest is the angles, read once per chunk); 31,000 tokens of 8 key heads
// in 16-token pages 120 us, 97%. By the chain of dependent loads (offsets,
// length, page id, rows) for a few tokens: 2.6 us for one, 4.2 us for 64
// sequences' next tokens, 6.5 us for 13 prompts of up to 360.
#include <algorithm>

#include "paged.cuh"
#include "sm103_ptx.cuh"

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
    long long units;
    int kv_chunks, chunks;  // chunks of key/value heads, and with the queries'
    int team;               // warps per unit
};

constexpr int kGroup = 16;  // slots per warp
// A warp's share of a token, by the warps that the call would have with four
// key heads each (of which 16 fit on an SM, 2,432 on 152): four heads, so that
// a token's angles serve eight rows, once that fills half of the places with
// whole groups of tokens (kWideFull) or all of them twice (kWideWarps, of which
// many have little to do); one head and two pairs of slots at once, more and
// shorter warps, while whole groups fill a quarter (kThinFull) and the other
// warps no more (kThinRest); two heads between. Measured (us, four / two / one):
// 20,400 tokens of 8 key heads with 4 queries each 91.9 / 102.5 / 134.7, 5,100
// of them 24.6 / 29.3 / 38.4, 2,500 17.4 / 14.7 / 20.0, 1,270 10.9 / 8.7 / 8.2;
// 1,480 tokens of 3 key heads 11.3 / 8.6 / 7.0; one token for each of 256
// sequences, 24 key heads, 13.9 / 16.0 / 27.5, of 64, 8 key heads, 6.9 / 4.5 /
// 6.0, of 8 6.3 / 3.9 / 3.4.
constexpr long long kWideFull = 1216, kWideWarps = 4864, kThinFull = 608, kThinRest = 700;

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

template <typename T> __device__ __forceinline__ void add8(float (&acc)[8], uint4 x) {
    const uint32_t r[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 e = unpack2<T>(r[j]);
        acc[2 * j] = __fadd_rn(acc[2 * j], e.x);
        acc[2 * j + 1] = __fadd_rn(acc[2 * j + 1], e.y);
    }
}

template <typename T, int HC, int PB>
__global__ void __launch_bounds__(512) k_paged_append(AppendArgs a) {
    extern __shared__ __align__(16) float ssum[];  // [units of the CTA][groups][HC][128] group sums
    const Paged &p = a.p;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, half = lane >> 4, i = lane & 15;
    const int groups = p.page / kGroup, per_cta = (int)(blockDim.x >> 5) / a.team;  // units per CTA
    const int chunk = (int)(blockIdx.x % a.chunks);         // neighbouring CTAs: the rows of the same tokens
    const int unit = wid / a.team, first_grp = wid % a.team;
    const long long u = (long long)(blockIdx.x / a.chunks) * per_cta + unit;
    const bool kv = chunk < a.kv_chunks;
    const T *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v), *q = static_cast<const T *>(a.q);
    T *kc = static_cast<T *>(a.kc), *vc = static_cast<T *>(a.vc), *qo = static_cast<T *>(a.q_out);
    grid_wait();

    // the unit: page `pg` of sequence b takes new tokens at slots [s0, s1)
    int b = 0, t_of = 0, s0 = 0, s1 = 0, pg = 0;  // slot s holds token t_of + s
    if (u < a.units) {
        int t0, n;
        if (a.cu) {
            b = find_seq(a, u, lane);
            t0 = cu_at(a, b);
            n = max(cu_at(a, b + 1) - t0, 0);
        } else {
            b = (int)u;
            t0 = b;
            n = 1;
        }
        const long long len = p.lens[b], first = len - n;  // unclamped: positions outside are dropped
        const long long lo = max(first, 0LL), hi = min(len, (long long)p.max_len);
        const long long base = a.cu ? (t0 >> p.page_log2) + 2LL * b : u;
        const long long pl = (lo >> p.page_log2) + (u - base);
        const long long at = pl << p.page_log2;
        if (n > 0 && lo < hi && at < hi) {
            pg = (int)pl;
            s0 = (int)max(lo - at, 0LL);
            s1 = (int)min(hi - at, (long long)p.page);
            t_of = (int)(t0 + (at - first));
        }
    }
    const bool work = s1 > s0;
    const int id = work && kv ? paged_id(p, b, pg) : -1;
    const bool mean = kv && a.mean && work && s1 == p.page && id >= 0;  // the page fills up in this call
    const long long page_at = (long long)max(id, 0) * p.page_stride;
    if (!kv) {
        const int h0 = (chunk - a.kv_chunks) * 2 * HC, hn = min(2 * HC, p.Hq - h0);
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
                if (fresh && 8 * i < a.rot) {
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
                    if (a.rot) x[c][h] = rotate<T>(a, x[c][h], w[c], i);
                    if (fresh && h < hn)
                        *reinterpret_cast<uint4 *>(qo + (tok * p.Hq + h0 + h) * kD + 8 * i) = x[c][h];
                }
            }
        }
        grid_go();
        return;
    }

    const int h0 = chunk * HC, hn = min(HC, p.Hkv - h0);
    for (int grp = first_grp; grp < groups; grp += a.team) {
        const int g0 = grp * kGroup;
        float acc[HC][8];
#pragma unroll
        for (int h = 0; h < HC; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[h][e] = 0.f;
        if (mean && g0 < s0) {  // the page's earlier keys, written by earlier calls
            constexpr int OB = HC <= 2 ? 8 / HC : 2;  // pairs of slots loaded together
            for (int st = 0; st < kGroup && g0 + st < s0; st += 2 * OB) {
                uint4 x[OB][HC];
#pragma unroll
                for (int c = 0; c < OB; ++c)
#pragma unroll
                    for (int h = 0; h < HC; ++h) {
                        const int s = g0 + st + 2 * c + half;
                        x[c][h] = s < s0 && h < hn ? *reinterpret_cast<const uint4 *>(kc + page_at + s * p.tok_stride +
                                                                                      (h0 + h) * p.head_stride + 8 * i)
                                                   : make_uint4(0, 0, 0, 0);  // adds nothing
                    }
#pragma unroll
                for (int c = 0; c < OB; ++c)
#pragma unroll
                    for (int h = 0; h < HC; ++h) add8<T>(acc[h], x[c][h]);
            }
        }
        if (g0 < s1 && g0 + kGroup > s0) {  // new tokens
            for (int st = 0; st < kGroup; st += 2 * PB) {
                if (g0 + st >= s1 || g0 + st + 2 * PB <= s0) continue;
                uint4 xk[PB][HC], xv[PB][HC];
                Angles w[PB];
#pragma unroll
                for (int c = 0; c < PB; ++c) {
                    const int s = g0 + st + 2 * c + half;
                    const bool fresh = s >= s0 && s < s1;
                    const long long tok = fresh ? t_of + s : 0;
#pragma unroll
                    for (int h = 0; h < HC; ++h) {
                        xk[c][h] = xv[c][h] = make_uint4(0, 0, 0, 0);
                        if (fresh && h < hn) {
                            xk[c][h] = *reinterpret_cast<const uint4 *>(k + tok * a.ks + (h0 + h) * kD + 8 * i);
                            xv[c][h] = *reinterpret_cast<const uint4 *>(v + tok * a.vs + (h0 + h) * kD + 8 * i);
                        }
                    }
                    if (fresh && 8 * i < a.rot) {
                        const int row = a.pos ? a.pos[tok] : (pg << p.page_log2) + s;
                        load_angles(a, clampi(row, 0, a.rows - 1), i, w[c]);
                    }
                }
#pragma unroll
                for (int c = 0; c < PB; ++c) {
                    const int s = g0 + st + 2 * c + half;
                    const bool fresh = s >= s0 && s < s1;
                    const long long slot_at = page_at + s * p.tok_stride + 8 * i;
#pragma unroll
                    for (int h = 0; h < HC; ++h) {
                        if (a.rot) xk[c][h] = rotate<T>(a, xk[c][h], w[c], i);
                        if (fresh && id >= 0 && h < hn) {
                            const long long at = slot_at + (h0 + h) * p.head_stride;
                            *reinterpret_cast<uint4 *>(kc + at) = xk[c][h];
                            *reinterpret_cast<uint4 *>(vc + at) = xv[c][h];
                        }
                        if (mean && fresh) add8<T>(acc[h], xk[c][h]);
                    }
                }
            }
        }
        if (mean)  // even + odd slots of the group
#pragma unroll
            for (int h = 0; h < HC; ++h)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float odd = __shfl_down_sync(0xffffffffu, acc[h][e], 16);
                    if (half == 0) ssum[((unit * groups + grp) * HC + h) * kD + 8 * i + e] = __fadd_rn(acc[h][e], odd);
                }
    }
    grid_go();
    if (!mean) return;
    ptx::named_sync(1 + unit, 32 * a.team);  // the unit's warps alone: others may have left
    if (first_grp == 0) {  // the groups in order
        const float inv = 1.f / (float)p.page;  // a power of two: exact
        for (int h = 0; h < hn; ++h) {
            float4 t = *reinterpret_cast<const float4 *>(&ssum[(unit * groups * HC + h) * kD + 4 * lane]);
            for (int g = 1; g < groups; ++g) {
                const float4 x = *reinterpret_cast<const float4 *>(&ssum[((unit * groups + g) * HC + h) * kD + 4 * lane]);
                t.x = __fadd_rn(t.x, x.x);
                t.y = __fadd_rn(t.y, x.y);
                t.z = __fadd_rn(t.z, x.z);
                t.w = __fadd_rn(t.w, x.w);
            }
            t.x *= inv, t.y *= inv, t.z *= inv, t.w *= inv;
            *reinterpret_cast<float4 *>(a.mean + ((long long)id * p.Hkv + h0 + h) * kD + 4 * lane) = t;
        }
    }
}

// Warps per unit: as many as a sequence's tokens fill groups on average (idle
// warps hold registers), and up to four for the earlier keys of a page that
// fills up.
int team_of(const AppendArgs &a) {
    const int groups = a.p.page / kGroup;
    int team = std::min(groups, 4);
    while (team < groups && (long long)a.T > (long long)team * kGroup * a.p.B) team *= 2;
    return team;
}

template <typename T, int HC, int PB> cudaError_t launch_append(AppendArgs &a, cudaStream_t s) {
    const int groups = a.p.page / kGroup;
    a.team = team_of(a);
    const int warps = a.team > 4 ? a.team : 4, per_cta = warps / a.team;
    a.kv_chunks = (a.p.Hkv + HC - 1) / HC;
    a.chunks = a.kv_chunks + (a.q ? (a.p.Hq + 2 * HC - 1) / (2 * HC) : 0);
    const long long ctas = (a.units + per_cta - 1) / per_cta * a.chunks;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const size_t smem = a.mean ? sizeof(float) * per_cta * groups * HC * kD : 0;
    return launch_paged(k_paged_append<T, HC, PB>, dim3((unsigned)ctas), 32 * warps, smem, 1, a, s);
}

}  // namespace
}  // namespace vsa

extern "C" vsa_status vsa_paged_append(const vsa_paged_desc *desc, int T, const void *k, int64_t k_stride,
                                       const void *v, int64_t v_stride, const void *q, int64_t q_stride, void *q_out,
                                       const int32_t *cu_seqlens, const int32_t *positions, const float *cos,
                                       const float *sin, int table_rows, int rot_dim, int interleaved, void *k_cache,
                                       void *v_cache, float *k_mean, vsa_stream_t stream) {
    using namespace vsa;
    AppendArgs a{};
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
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    prof_begin("paged_append", s);
    const bool bf = a.p.dtype == T_BF16;
    const long long chunks = (a.p.Hkv + 3) / 4 + (q ? (a.p.Hq + 7) / 8 : 0), warps = a.units * team_of(a) * chunks;
    const long long full = T / kGroup * chunks;
    const bool wide = full > kWideFull || warps > kWideWarps, thin = full <= kThinFull && warps - full <= kThinRest;
    const cudaError_t e = wide   ? (bf ? launch_append<__nv_bfloat16, 4, 1>(a, s) : launch_append<__half, 4, 1>(a, s))
                          : thin ? (bf ? launch_append<__nv_bfloat16, 1, 2>(a, s) : launch_append<__half, 1, 2>(a, s))
                                 : (bf ? launch_append<__nv_bfloat16, 2, 1>(a, s) : launch_append<__half, 2, 1>(a, s));
    prof_end(s);
    return status_from_cuda(e);
}
