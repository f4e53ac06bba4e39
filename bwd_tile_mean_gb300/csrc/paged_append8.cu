// paged_append8.cu -- vsa_paged8_append: new tokens' keys and values into a
// paged cache of e4m3 bytes with a scale per block of 16 tokens and key/value
// head, keys and queries rotated on the way, means of pages that fill up; and
// vsa_paged_read, the way back.
//
// A block's scale is the least power of two that brings the largest entry
// within 448. A power of two, since e4m3 floats anyway: a full-precision scale
// would win at most one of its exponents, and would round the block's earlier
// tokens again whenever a later one raised it. So, when a token arrives whose
// entries need a larger scale, the earlier ones are multiplied by a power of
// two: their bits stay the same four significant ones but for what falls below
// 2^-6 of the new scale, e4m3's subnormals, which round a second time. A block
// whose first slot is written starts afresh, whatever its bytes held before.
//
// The units of work are those of the 16-bit append (paged_rows.cuh). A 16-slot
// group of a unit is a block, held by one warp for one head after another: half
// a warp per token row, 8 dims per lane, all of the block's rotated keys in
// registers in fp32 (they are rounded once, to e4m3) until its largest entry is
// known.
#include "e4m3.cuh"
#include "paged_rows.cuh"
#include "sm103_ptx.cuh"

namespace vsa {
namespace {

// The lane's 8 dims of a key, rotated, in fp32; whole warp.
template <typename T>
__device__ __forceinline__ void rotate8(const AppendArgs &a, uint4 x, const Angles &w, int i, float (&y)[8]) {
    const uint32_t r[4] = {x.x, x.y, x.z, x.w};
    const int hop = a.rot >> 4;
    const bool on = 8 * i < a.rot, lower = i < hop;
    const int peer = (threadIdx.x & 16) | (on ? (lower ? i + hop : i - hop) : i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 e = unpack2<T>(r[j]);
        y[2 * j] = e.x;
        y[2 * j + 1] = e.y;
        if (a.rot == 0) continue;
        if (a.inter) {
            if (on) {
                y[2 * j] = __fsub_rn(__fmul_rn(e.x, w.c[j]), __fmul_rn(e.y, w.s[j]));
                y[2 * j + 1] = __fadd_rn(__fmul_rn(e.y, w.c[j]), __fmul_rn(e.x, w.s[j]));
            }
        } else {
            const float2 f = unpack2<T>(__shfl_sync(0xffffffffu, r[j], peer));
            if (on) {
                const float sx = lower ? -w.s[2 * j] : w.s[2 * j], sy = lower ? -w.s[2 * j + 1] : w.s[2 * j + 1];
                y[2 * j] = __fadd_rn(__fmul_rn(e.x, w.c[2 * j]), __fmul_rn(f.x, sx));
                y[2 * j + 1] = __fadd_rn(__fmul_rn(e.y, w.c[2 * j + 1]), __fmul_rn(f.y, sy));
            }
        }
    }
}

// What dtype holds: entries that are infinite in it do not fit, and no byte may stand for more than its largest value: 256
// times the largest scale would (65,536, and 2^128).
template <typename T> struct Range;
template <> struct Range<__nv_bfloat16> {
    static __device__ __forceinline__ bool fits(float x) { return fabsf(x) < INFINITY; }
    static __device__ __forceinline__ float most(float scale) { return scale == 0x1p120f ? 240.f : 448.f; }
};
template <> struct Range<__half> {
    static __device__ __forceinline__ bool fits(float x) { return fabsf(x) < 65520.f; }
    static __device__ __forceinline__ float most(float scale) { return scale == 256.f ? 240.f : 448.f; }
};
template <typename T> __device__ __forceinline__ float top_of(const float (&x)[8], float top) {
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, Range<T>::fits(x[e]) ? fabsf(x[e]) : 0.f);
    return top;
}
__device__ __forceinline__ float warp_top(float x) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    return x;
}
// 8 entries as bytes of this scale (inv: its inverse); infinities as NaN.
template <typename T> __device__ __forceinline__ uint2 bytes_of(const float (&x)[8], float scale, float inv) {
    const float most = Range<T>::most(scale);
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float v = x[2 * j + e];
            y[e] = Range<T>::fits(v) ? fminf(fmaxf(v * inv, -most), most) : __int_as_float(0x7fffffff);
        }
        r[j] = e4m3x2_of(y[0], y[1]);
    }
    return make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
}
__device__ __forceinline__ void floats_of(uint2 b, float scale, float (&y)[8]) {
    const uint32_t r[4] = {b.x, b.x >> 16, b.y, b.y >> 16};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = float2_of(r[j]);
        y[2 * j] = v.x * scale;
        y[2 * j + 1] = v.y * scale;
    }
}
__device__ __forceinline__ void add8(float (&acc)[8], uint2 b, float scale) {
    float y[8];
    floats_of(b, scale, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = __fadd_rn(acc[e], y[e]);
}
template <typename T> __device__ __forceinline__ void unpack8(uint4 x, float (&y)[8]) {
    const uint32_t r[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = unpack2<T>(r[j]);
        y[2 * j] = v.x;
        y[2 * j + 1] = v.y;
    }
}

constexpr int kPairs = kGroup / 2;  // pairs of slots of a block: one of each for every half of the warp

// HC, PB: the queries' heads (2 HC) and pairs of slots at once; a.hc key/value heads per chunk.
template <typename T, int HC, int PB> __global__ void __launch_bounds__(256) k_paged8_append(AppendArgs a) {
    extern __shared__ __align__(16) float ssum[];  // [units of the CTA][groups][hc][128] group sums
    const Paged &p = a.p;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, half = lane >> 4, i = lane & 15;
    const int groups = p.page / kGroup, per_cta = (int)(blockDim.x >> 5) / a.team;
    const int chunk = (int)(blockIdx.x % a.chunks);
    const int unit = wid / a.team, first_grp = wid % a.team;
    const long long u = (long long)(blockIdx.x / a.chunks) * per_cta + unit;
    const T *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v);
    unsigned char *kc = static_cast<unsigned char *>(a.kc), *vc = static_cast<unsigned char *>(a.vc);
    grid_wait();

    const Unit of = find_unit(a, u, lane);
    const int s0 = of.s0, s1 = of.s1;
    if (chunk >= a.kv_chunks) {
        append_queries<T, HC, PB>(a, of, (chunk - a.kv_chunks) * 2 * HC, first_grp);
        grid_go();
        return;
    }
    const int id = s1 > s0 ? paged_id(p, of.b, of.pg) : -1;
    const bool mean = a.mean && s1 == p.page && id >= 0;  // the page fills up in this call
    const long long page_at = (long long)max(id, 0) * p.page_stride + 8 * i;
    const int h0 = chunk * a.hc, hn = min(a.hc, p.Hkv - h0);
    for (int grp = first_grp; grp < groups && id >= 0; grp += a.team) {
        const int g0 = grp * kGroup;
        const bool fresh = g0 < s1 && g0 + kGroup > s0, begun = g0 < s0;
        if (!fresh && !(mean && begun)) continue;
        for (int hh = 0; hh < hn; ++hh) {
            const int h = h0 + hh;
            const long long at = page_at + h * p.head_stride, sc = ((long long)id * p.Hkv + h) * groups + grp;
            const float k_old = begun ? a.kscale[sc] : 0.f, v_old = begun && fresh ? a.vscale[sc] : 0.f;
            float ks = k_old, vs = v_old;
            float key[kPairs][8];
            uint4 xv[kPairs];
            if (fresh) {
                uint4 xk[kPairs];
#pragma unroll
                for (int c = 0; c < kPairs; ++c) {
                    const int s = g0 + 2 * c + half;
                    xk[c] = xv[c] = make_uint4(0, 0, 0, 0);
                    if (s >= s0 && s < s1) {
                        const long long tok = of.t_of + s;
                        xk[c] = *reinterpret_cast<const uint4 *>(k + tok * a.ks + h * kD + 8 * i);
                        xv[c] = *reinterpret_cast<const uint4 *>(v + tok * a.vs + h * kD + 8 * i);
                    }
                }
                float k_top = 0.f, v_top = 0.f;
#pragma unroll
                for (int c = 0; c < kPairs; ++c) {
                    if (g0 + 2 * c + 1 < s0 || g0 + 2 * c >= s1) continue;
                    const int s = g0 + 2 * c + half;
                    Angles w;
                    if (8 * i < a.rot && s >= s0 && s < s1) {
                        const int row = a.pos ? a.pos[of.t_of + s] : (of.pg << p.page_log2) + s;
                        load_angles(a, clampi(row, 0, a.rows - 1), i, w);
                    }
                    rotate8<T>(a, xk[c], w, i, key[c]);
                    float val[8];
                    unpack8<T>(xv[c], val);
                    if (s >= s0 && s < s1) {
                        k_top = top_of<T>(key[c], k_top);
                        v_top = top_of<T>(val, v_top);
                    }
                }
                ks = fmaxf(scale_of(warp_top(k_top)), k_old);
                vs = fmaxf(scale_of(warp_top(v_top)), v_old);
            }
            float acc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.f;
            const bool k_grown = begun && ks != k_old, v_grown = begun && fresh && vs != v_old;
            if (begun && (mean || k_grown || v_grown)) {  // the block's earlier tokens
                const float k_by = k_old / ks, v_by = v_grown ? v_old / vs : 1.f;
#pragma unroll
                for (int c = 0; c < kPairs; ++c) {
                    const int s = g0 + 2 * c + half;
                    if (s >= s0) continue;
                    unsigned char *ka = kc + at + s * p.tok_stride, *va = vc + at + s * p.tok_stride;
                    if (k_grown || mean) {
                        uint2 b = *reinterpret_cast<const uint2 *>(ka);
                        if (k_grown) {
                            float y[8];
                            floats_of(b, k_by, y);
                            b = make_uint2(e4m3x2_of(y[0], y[1]) | e4m3x2_of(y[2], y[3]) << 16,
                                           e4m3x2_of(y[4], y[5]) | e4m3x2_of(y[6], y[7]) << 16);
                            *reinterpret_cast<uint2 *>(ka) = b;
                        }
                        if (mean) add8(acc, b, ks);
                    }
                    if (v_grown) {
                        float y[8];
                        floats_of(*reinterpret_cast<const uint2 *>(va), v_by, y);
                        *reinterpret_cast<uint2 *>(va) = make_uint2(e4m3x2_of(y[0], y[1]) | e4m3x2_of(y[2], y[3]) << 16,
                                                                    e4m3x2_of(y[4], y[5]) | e4m3x2_of(y[6], y[7]) << 16);
                    }
                }
            }
            if (fresh) {
                const float k_inv = 1.f / ks, v_inv = 1.f / vs;
#pragma unroll
                for (int c = 0; c < kPairs; ++c) {
                    const int s = g0 + 2 * c + half;
                    if (s < s0 || s >= s1) continue;
                    float val[8];
                    unpack8<T>(xv[c], val);
                    const uint2 b = bytes_of<T>(key[c], ks, k_inv);
                    *reinterpret_cast<uint2 *>(kc + at + s * p.tok_stride) = b;
                    *reinterpret_cast<uint2 *>(vc + at + s * p.tok_stride) = bytes_of<T>(val, vs, v_inv);
                    if (mean) add8(acc, b, ks);
                }
                if (lane == 0) {
                    a.kscale[sc] = ks;
                    a.vscale[sc] = vs;
                }
            }
            if (mean)  // even + odd slots of the group
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float odd = __shfl_down_sync(0xffffffffu, acc[e], 16);
                    if (half == 0) ssum[((unit * groups + grp) * a.hc + hh) * kD + 8 * i + e] = __fadd_rn(acc[e], odd);
                }
        }
    }
    grid_go();
    if (!mean) return;
    ptx::named_sync(1 + unit, 32 * a.team);  // the unit's warps alone: others may have left
    if (first_grp == 0) {  // the groups in order
        const float inv = 1.f / (float)p.page;  // a power of two: exact
        for (int hh = 0; hh < hn; ++hh) {
            float4 t = *reinterpret_cast<const float4 *>(&ssum[(unit * groups * a.hc + hh) * kD + 4 * lane]);
            for (int g = 1; g < groups; ++g) {
                const float4 x = *reinterpret_cast<const float4 *>(&ssum[((unit * groups + g) * a.hc + hh) * kD + 4 * lane]);
                t.x = __fadd_rn(t.x, x.x);
                t.y = __fadd_rn(t.y, x.y);
                t.z = __fadd_rn(t.z, x.z);
                t.w = __fadd_rn(t.w, x.w);
            }
            t.x *= inv, t.y *= inv, t.z *= inv, t.w *= inv;
            *reinterpret_cast<float4 *>(a.mean + ((long long)id * p.Hkv + h0 + hh) * kD + 4 * lane) = t;
        }
    }
}

template <typename T, int HC, int PB> cudaError_t launch_append8(AppendArgs &a, cudaStream_t s) {
    const int groups = a.p.page / kGroup;
    a.team = std::min(team_of(a), 8);
    const int warps = a.team > 4 ? a.team : 4, per_cta = warps / a.team;
    a.hc = HC;
    a.kv_chunks = (a.p.Hkv + a.hc - 1) / a.hc;
    a.chunks = a.kv_chunks + (a.q ? (a.p.Hq + 2 * HC - 1) / (2 * HC) : 0);
    const long long ctas = (a.units + per_cta - 1) / per_cta * a.chunks;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const size_t smem = a.mean ? sizeof(float) * per_cta * groups * a.hc * kD : 0;
    return launch_paged(k_paged8_append<T, HC, PB>, dim3((unsigned)ctas), 32 * warps, smem, 1, a, s);
}

struct ReadArgs {
    Paged p;
    int T;
    const int *cu;
    const void *kc, *vc;
    const float *ks, *vs;  // 8 bits
    void *k, *v;
    int chunk, chunks;     // heads per warp, warps per token
};

// The stored values of tokens, as dtype: a warp has one token and a chunk of its heads, half of it keys, the other half
// values; 8 dims per lane.
template <typename T, int KV> __global__ void __launch_bounds__(256) k_paged_read(ReadArgs a) {
    const Paged &p = a.p;
    const int lane = threadIdx.x & 31, half = lane >> 4, i = lane & 15;
    grid_wait();
    const long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t = (int)(u / a.chunks), h0 = (int)(u % a.chunks) * a.chunk, h1 = min(h0 + a.chunk, p.Hkv);
    if (t >= a.T) return;
    int b = t;
    long long pos;
    if (a.cu) {
        // the last sequence with cu[b] <= t
        int lo = 0, n = p.B;
        while (n > 1) {
            const int step = (n + 31) >> 5, at = lo + lane * step;
            const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && clampi(a.cu[at], 0, a.T) <= t);
            const int last = m ? 31 - __clz(m) : 0, end = lo + n;
            lo += last * step;
            n = min(step, end - lo);
        }
        b = lo;
        const int t1 = clampi(a.cu[b + 1], 0, a.T);
        if (t < clampi(a.cu[b], 0, a.T) || t >= t1) return;  // behind the last sequence
        pos = (long long)p.lens[b] - (t1 - t);
    } else {
        pos = (long long)p.lens[b] - 1;
    }
    const int id = pos >= 0 && pos < p.max_len ? paged_id(p, b, (int)(pos >> p.page_log2)) : -1;
    const int slot = (int)(pos & (p.page - 1));
    T *to = static_cast<T *>(half ? a.v : a.k) + (long long)t * p.Hkv * kD + 8 * i;
    const long long from = (long long)max(id, 0) * p.page_stride + slot * p.tok_stride + 8 * i;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (id >= 0) {
            if constexpr (KV == 8) {
                const unsigned char *c = static_cast<const unsigned char *>(half ? a.vc : a.kc);
                const uint2 w = *reinterpret_cast<const uint2 *>(c + from + h * p.head_stride);
                float y[8];
                floats_of(w, (half ? a.vs : a.ks)[((long long)id * p.Hkv + h) * (p.page / kGroup) + slot / kGroup], y);
                x = make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
            } else {
                x = *reinterpret_cast<const uint4 *>(static_cast<const T *>(half ? a.vc : a.kc) + from + h * p.head_stride);
            }
        }
        *reinterpret_cast<uint4 *>(to + (long long)h * kD) = x;
    }
    grid_go();
}

}  // namespace
}  // namespace vsa

using namespace vsa;

extern "C" vsa_status vsa_paged8_append(const vsa_paged_desc *desc, int T, const void *k, int64_t k_stride, const void *v,
                                        int64_t v_stride, const void *q, int64_t q_stride, void *q_out,
                                        const int32_t *cu_seqlens, const int32_t *positions, const float *cos,
                                        const float *sin, int table_rows, int rot_dim, int interleaved, void *k_cache,
                                        void *v_cache, float *k_scale, float *v_scale, float *k_mean, vsa_stream_t stream) {
    AppendArgs a{};
    const vsa_status st = append_args(desc, T, k, k_stride, v, v_stride, q, q_stride, q_out, cu_seqlens, positions, cos, sin,
                                      table_rows, rot_dim, interleaved, k_cache, v_cache, k_mean, &a);
    if (st != VSA_OK) return st;
    if (a.p.page_stride % 16 != 0) return VSA_ERR_SHAPE;
    if (!k_scale || !v_scale) return VSA_ERR_NULL;
    if (((uintptr_t)k_scale | (uintptr_t)v_scale) & 3u) return VSA_ERR_LAYOUT;
    if (T == 0) return VSA_OK;
    a.kscale = k_scale;
    a.vscale = v_scale;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    prof_begin("paged8_append", s);
    const bool bf = a.p.dtype == T_BF16;
    const long long chunks = (a.p.Hkv + 3) / 4 + (q ? (a.p.Hq + 7) / 8 : 0), full = T / kGroup * chunks;
    const cudaError_t e = full > 1216 ? (bf ? launch_append8<__nv_bfloat16, 4, 1>(a, s) : launch_append8<__half, 4, 1>(a, s))
                                      : (bf ? launch_append8<__nv_bfloat16, 1, 2>(a, s) : launch_append8<__half, 1, 2>(a, s));
    prof_end(s);
    return status_from_cuda(e);
}

extern "C" vsa_status vsa_paged_read(const vsa_paged_desc *desc, int T, const int32_t *cu_seqlens, const void *k_cache,
                                     const void *v_cache, const float *k_scale, const float *v_scale, void *k_out, void *v_out,
                                     vsa_stream_t stream) {
    ReadArgs a{};
    const vsa_status st = to_paged(desc, &a.p, true);
    if (st != VSA_OK) return st;
    if (T < 0 || (!cu_seqlens && T != a.p.B)) return VSA_ERR_SHAPE;
    if (!k_cache || !v_cache || !k_scale != !v_scale) return VSA_ERR_NULL;
    const bool eight = k_scale != nullptr;
    if (eight && a.p.page_stride % 16 != 0) return VSA_ERR_SHAPE;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out)) return VSA_ERR_LAYOUT;
    if (((uintptr_t)cu_seqlens | (uintptr_t)k_scale | (uintptr_t)v_scale) & 3u) return VSA_ERR_LAYOUT;
    if (T == 0) return VSA_OK;
    if (!k_out || !v_out) return VSA_ERR_NULL;
    a.T = T;
    a.cu = cu_seqlens;
    a.kc = k_cache;
    a.vc = v_cache;
    a.ks = k_scale;
    a.vs = v_scale;
    a.k = k_out;
    a.v = v_out;
    // all heads of a token in one warp, or as many warps as fill the GPU
    const long long split = std::min<long long>(a.p.Hkv, std::max(1LL, 152LL * 32 / T));
    a.chunk = (int)((a.p.Hkv + split - 1) / split);
    a.chunks = (a.p.Hkv + a.chunk - 1) / a.chunk;
    const long long ctas = ((long long)T * a.chunks + 7) / 8;
    if (ctas > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    prof_begin("paged_read", s);
    const bool bf = a.p.dtype == T_BF16;
    const auto kernel = eight ? (bf ? k_paged_read<__nv_bfloat16, 8> : k_paged_read<__half, 8>)
                              : (bf ? k_paged_read<__nv_bfloat16, 16> : k_paged_read<__half, 16>);
    const cudaError_t e = launch_paged(kernel, dim3((unsigned)ctas), 256, 0, 1, a, s);
    prof_end(s);
    return status_from_cuda(e);
}
