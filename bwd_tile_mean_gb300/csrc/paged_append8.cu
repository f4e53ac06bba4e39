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
// group of a unit is a block, taken by one warp for one head after another: half
// a warp per token row, 8 dims per lane.
//
// Bound by instructions for long prompts: 30,000 tokens of 24 heads (0.92 GB) take
// 204 us, 66% of the measured copy rate, with 54% of the issue slots and 58% of
// DRAM's peak busy (half style, whose pairs lie in two lanes, a fifth more); the
// blocks are rotated, searched and rounded in fp32. Measured on the way there, each
// with what was built then (us): rotated keys kept in registers, 8 warps per SM 360; with
// 128 registers and spills 377; walked twice from shared memory 266, two heads per
// warp 248 (one 272, four 266), with angles by position 207, loops unrolled four deep
// 203 (two 207, one 221); a head instead of a group per warp, which share their
// angles, 225. Reading the same tokens back (0.55 GB) 96 us, 85%. One token for each
// of 64 sequences, 8 key heads: 6 us, the chain length, page id, scale, two walks,
// and the earlier keys of a page that fills up.
#include <type_traits>

#include "e4m3.cuh"
#include "paged_rows.cuh"
#include "sm103_ptx.cuh"

namespace vsa {
namespace {

// The lane's 8 dims of a key, rotated, in fp32; whole warp. peer: the lane with the other dims of its pairs.
template <typename T, bool kInter, bool kAll>
__device__ __forceinline__ void rotate8(uint4 x, const Angles &w, bool on, bool lower, int peer, float (&y)[8]) {
    const uint32_t r[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 e = unpack2<T>(r[j]);
        float u, v;
        if constexpr (kInter) {
            u = __fsub_rn(__fmul_rn(e.x, w.c[j]), __fmul_rn(e.y, w.s[j]));
            v = __fadd_rn(__fmul_rn(e.y, w.c[j]), __fmul_rn(e.x, w.s[j]));
        } else {
            // lower dims: x1 c + (-x2) s, the same bits as x1 c - x2 s. (Paired multiplications and additions become fused
            // ones, which round once.)
            const float2 f = unpack2<T>(__shfl_sync(0xffffffffu, r[j], peer) ^ (lower ? 0x80008000u : 0u));
            u = __fadd_rn(__fmul_rn(e.x, w.c[2 * j]), __fmul_rn(f.x, w.s[2 * j]));
            v = __fadd_rn(__fmul_rn(e.y, w.c[2 * j + 1]), __fmul_rn(f.y, w.s[2 * j + 1]));
        }
        y[2 * j] = kAll || on ? u : e.x;
        y[2 * j + 1] = kAll || on ? v : e.y;
    }
}

// What dtype holds: entries that are infinite in it do not fit, and no byte may stand for more than its largest value: 256
// times the largest scale would (65,536, and 2^128).
template <typename T> struct Range;
template <> struct Range<__nv_bfloat16> {
    static constexpr float kInf = INFINITY, kTop = 0x1p120f;
};
template <> struct Range<__half> {
    static constexpr float kInf = 65520.f, kTop = 256.f;
};
// Largest magnitude of 8 entries and `top`; NaN does not count.
__device__ __forceinline__ float top_of(const float (&x)[8], float top) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) top = ptx::fmax3(top, fabsf(x[e]), fabsf(x[e + 1]));
    return top;
}
// ... of those that fit.
template <typename T> __device__ __forceinline__ float top_fitting(const float (&x)[8], float top) {
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]) < Range<T>::kInf ? fabsf(x[e]) : 0.f);
    return top;
}
__device__ __forceinline__ float warp_top(float x) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    return x;
}
// 8 entries as bytes of a scale, by its inverse. `plain`: all fit, and the scale is below the largest; otherwise infinities
// become NaN, and others the largest value that the scale brings within dtype: 240 (1.875 2^7) for the largest scale that is
// made here, less in steps of 2^-9 at the end for a larger one that the cache came with.
template <typename T> __device__ __forceinline__ uint2 bytes_of(const float (&x)[8], float inv, bool plain) {
    uint32_t r[4];
    if (plain) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 y = ptx::f32x2_split(ptx::fmul_x2(ptx::f32x2(x[2 * j], x[2 * j + 1]), ptx::f32x2(inv, inv)));
            r[j] = e4m3x2_of(y.x, y.y);
        }
    } else {
        const float top = 240.f * (Range<T>::kTop * inv);
        const float most = top > 240.f ? 448.f : top < 0x1p-6f ? floorf(top * 0x1p9f) * 0x1p-9f : top;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float v = x[2 * j + e];
                y[e] = fabsf(v) < Range<T>::kInf ? fminf(fmaxf(v * inv, -most), most) : __int_as_float(0x7fffffff);
            }
            r[j] = e4m3x2_of(y[0], y[1]);
        }
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
// Adds what the bytes stand for over their scale, a power of two: the sums have the bits of those of the values.
__device__ __forceinline__ void add8(float (&acc)[8], uint2 b) {
    const uint32_t r[4] = {b.x, b.x >> 16, b.y, b.y >> 16};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = float2_of(r[j]);
        const float2 sum = ptx::f32x2_split(ptx::fadd_x2(ptx::f32x2(acc[2 * j], acc[2 * j + 1]), ptx::f32x2(v.x, v.y)));
        acc[2 * j] = sum.x;
        acc[2 * j + 1] = sum.y;
    }
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
constexpr int kRawBytes = kPairs * 512;  // a block's keys, or values, as they come

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 own16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// Largest magnitudes of two packed rows of 8 entries, NaN apart.
template <typename T> __device__ __forceinline__ uint32_t top2(uint4 x, uint32_t top) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const uint32_t r[4] = {x.x, x.y, x.z, x.w};
    T2 t = *reinterpret_cast<const T2 *>(&top);
#pragma unroll
    for (int j = 0; j < 4; ++j) t = __hmax2(t, __habs2(*reinterpret_cast<const T2 *>(&r[j])));
    return *reinterpret_cast<const uint32_t *>(&t);
}

// HC, PB: the queries' heads (2 HC) and pairs of slots at once; a.hc key/value heads per chunk. A warp's next block comes
// into its part of shared memory (values, keys; a lane reads back what it copied itself) while it works on one, and is
// walked twice: for the largest entry, and to be rounded. Rotating twice takes fewer instructions than it takes registers to
// keep 64 rotated entries per lane. kAll: all dims are rotated, by the tokens' positions themselves. kFew: for calls
// of few tokens, whose time is their code's way into the instruction caches.
template <typename T, bool kInter, bool kAll, int HC, int PB, bool kFew>
__global__ void __launch_bounds__(256, 2) k_paged8_append(AppendArgs a) {
    constexpr int kUnroll = kFew ? 1 : 4;
    extern __shared__ __align__(16) unsigned char smem[];  // [warps][2][kRawBytes], [units of the CTA][groups][hc][128] sums
    const Paged &p = a.p;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, half = lane >> 4, i = lane & 15, warps = (int)(blockDim.x >> 5);
    float *ssum = reinterpret_cast<float *>(smem + warps * 2 * kRawBytes);
    const uint32_t raw_v = ptx::smem_addr(smem) + wid * 2 * kRawBytes + lane * 16, raw_k = raw_v + kRawBytes;
    const int groups = p.page / kGroup, per_cta = warps / a.team;
    const int chunk = (int)(blockIdx.x % a.chunks);
    const int unit = wid / a.team, first_grp = wid % a.team;
    const long long u = (long long)(blockIdx.x / a.chunks) * per_cta + unit;
    grid_wait();

    const Unit of = find_unit(a, u, lane);
    const int s0 = of.s0, s1 = of.s1;
    if (chunk >= a.kv_chunks) {
        const int part = chunk - a.kv_chunks;
        append_queries<T, HC, PB, !kAll ? 0 : kInter ? 1 : 2>(a, of, (a.single ? part * a.team + first_grp : part) * 2 * HC,
                                                              a.single ? s0 / kGroup : first_grp);
        grid_go();
        return;
    }
    const int id = s1 > s0 ? paged_id(p, of.b, of.pg) : -1;
    const bool mean = a.mean && s1 == p.page;  // the page fills up in this call
    const int h0 = chunk * a.hc, hn = min(a.hc, p.Hkv - h0);
    const long long page_at = (long long)max(id, 0) * p.page_stride + half * p.tok_stride + 8 * i;
    const int hop = a.rot >> 4;  // half style: lanes from a dim to the other of its pair
    const bool on = kAll || 8 * i < a.rot, lower = i < hop;
    const int peer = kAll ? lane ^ 8 : (threadIdx.x & 16) | (on ? (lower ? i + hop : i - hop) : i);
    const int first_row = of.pg << p.page_log2;
    // a lane has slot g0 + 2 c + half of block grp at pair c: the new ones are copied
    auto copy = [&](const void *base, long long stride, uint32_t dst, int grp, int hh) {
        const int s = grp * kGroup + half;
        const T *from = static_cast<const T *>(base) + ((long long)of.t_of + s) * stride + (h0 + hh) * kD + 8 * i;
#pragma unroll
        for (int c = 0; c < kPairs; ++c)
            if (s + 2 * c >= s0 && s + 2 * c < s1) copy16(dst + c * 512, from + 2 * c * stride);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto no_copy = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    auto has_new = [&](int grp) { return grp < groups && grp * kGroup < s1 && grp * kGroup + kGroup > s0; };
    auto skip = [&](int grp) { return grp < groups && !has_new(grp) && !(mean && grp * kGroup < s0); };
    int grp = first_grp, hh = 0;
    while (skip(grp)) grp += a.team;
    if (has_new(grp)) {
        copy(a.v, a.vs, raw_v, grp, hh);
        copy(a.k, a.ks, raw_k, grp, hh);
        if (id < 0) asm volatile("cp.async.wait_group 0;" ::: "memory");  // nothing to store: the copies do not outlive the warp
    }
    while (id >= 0 && grp < groups) {
        const int g0 = grp * kGroup, h = h0 + hh, mine = g0 + half;
        const bool fresh = has_new(grp), begun = g0 < s0;
        int grp1 = grp, hh1 = hh + 1;  // the next block
        if (hh1 == hn) {
            hh1 = 0;
            do grp1 += a.team;
            while (skip(grp1));
        }
        const bool more = has_new(grp1);
        const long long sc = ((long long)id * p.Hkv + h) * groups + grp;
        unsigned char *kc = static_cast<unsigned char *>(a.kc) + page_at + h * p.head_stride + g0 * p.tok_stride;
        unsigned char *vc = static_cast<unsigned char *>(a.vc) + page_at + h * p.head_stride + g0 * p.tok_stride;
        const float k_old = begun ? a.kscale[sc] : 0.f, v_old = begun && fresh ? a.vscale[sc] : 0.f;
        float ks = k_old;
        const int c0 = max(s0 - g0, 0) >> 1, c1 = (min(s1 - g0, kGroup) + 1) >> 1;  // pairs with new slots
        auto is_new = [&](int c) { return mine + 2 * c >= s0 && mine + 2 * c < s1; };
        // earlier tokens of the block, `by` times what they are
        auto shrink = [&](unsigned char *at, float by) {
#pragma unroll 1
            for (int c = 0; c < kPairs; ++c) {
                if (mine + 2 * c >= s0) break;
                uint2 *to = reinterpret_cast<uint2 *>(at + 2 * c * p.tok_stride);
                float y[8];
                floats_of(*to, by, y);
                *to = make_uint2(e4m3x2_of(y[0], y[1]) | e4m3x2_of(y[2], y[3]) << 16,
                                 e4m3x2_of(y[4], y[5]) | e4m3x2_of(y[6], y[7]) << 16);
            }
        };
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        auto old_keys = [&] {  // of a page that fills up, at their final scale
#pragma unroll 4
            for (int c = 0; c < kPairs; ++c) {
                if (mine + 2 * c >= s0) break;
                add8(acc, *reinterpret_cast<const uint2 *>(kc + 2 * c * p.tok_stride));
            }
        };
        if (fresh) {
            {   // values
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                auto value = [&](int c) { return is_new(c) ? own16(raw_v + c * 512) : make_uint4(0, 0, 0, 0); };
                uint32_t t2 = 0;
#pragma unroll kUnroll
                for (int c = c0; c < c1; ++c) t2 = top2<T>(value(c), t2);
                const float2 t = unpack2<T>(t2);
                float top = warp_top(fmaxf(t.x, t.y));
                bool plain = top < Range<T>::kInf;
                if (!plain) {
                    top = 0.f;
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {
                        float y[8];
                        unpack8<T>(value(c), y);
                        top = top_fitting<T>(y, top);
                    }
                    top = warp_top(top);
                }
                const float vs = fmaxf(scale_of(top), v_old), inv = 1.f / vs;
                plain = plain && vs < Range<T>::kTop;
                if (begun && vs != v_old) shrink(vc, v_old / vs);
#pragma unroll kUnroll
                for (int c = c0; c < c1; ++c) {
                    float y[8];
                    unpack8<T>(value(c), y);
                    if (is_new(c)) *reinterpret_cast<uint2 *>(vc + 2 * c * p.tok_stride) = bytes_of<T>(y, inv, plain);
                }
                if (lane == 0) a.vscale[sc] = vs;
                if (more)
                    copy(a.v, a.vs, raw_v, grp1, hh1);
                else
                    no_copy();
            }
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            auto key = [&](int c, float (&y)[8]) {
                const bool in = is_new(c);
                Angles w;
                if constexpr (kAll) {  // of slots that are not new too: times 0
                    const int row = min(first_row + mine + 2 * c, a.rows - 1);
                    const long long at = (long long)row * 64 + (kInter ? 4 * i : 8 * (i & 7));
                    load4(w.c, a.cos + at);
                    load4(w.s, a.sin + at);
                    if constexpr (!kInter) {
                        load4(w.c + 4, a.cos + at + 4);
                        load4(w.s + 4, a.sin + at + 4);
                    }
                } else if (on) {
                    const int s = mine + 2 * c, row = !in ? 0 : a.pos ? a.pos[of.t_of + s] : first_row + s;
                    load_angles(a, clampi(row, 0, a.rows - 1), i, w);
                }
                rotate8<T, kInter, kAll>(in ? own16(raw_k + c * 512) : make_uint4(0, 0, 0, 0), w, on, lower, peer, y);
            };
            float top = 0.f;
#pragma unroll kUnroll
            for (int c = c0; c < c1; ++c) {
                float y[8];
                key(c, y);
                top = top_of(y, top);
            }
            top = warp_top(top);
            bool plain = top < Range<T>::kInf;
            if (!plain) {
                top = 0.f;
#pragma unroll 1
                for (int c = c0; c < c1; ++c) {
                    float y[8];
                    key(c, y);
                    top = top_fitting<T>(y, top);
                }
                top = warp_top(top);
            }
            ks = fmaxf(scale_of(top), k_old);
            plain = plain && ks < Range<T>::kTop;
            const float inv = 1.f / ks;
            if (begun && ks != k_old) shrink(kc, k_old / ks);
            if (mean && begun) old_keys();
#pragma unroll kUnroll
            for (int c = c0; c < c1; ++c) {
                float y[8];
                key(c, y);
                const uint2 b = bytes_of<T>(y, inv, plain);
                if (is_new(c)) {
                    *reinterpret_cast<uint2 *>(kc + 2 * c * p.tok_stride) = b;
                    if (mean) add8(acc, b);
                }
            }
            if (more)
                copy(a.k, a.ks, raw_k, grp1, hh1);
            else
                no_copy();
            if (lane == 0) a.kscale[sc] = ks;
        } else {
            old_keys();
            if (more) {  // a block of earlier tokens alone is followed by one with new ones
                copy(a.v, a.vs, raw_v, grp1, hh1);
                copy(a.k, a.ks, raw_k, grp1, hh1);
            }
        }
        if (mean)  // even + odd slots of the group
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float odd = __shfl_down_sync(0xffffffffu, acc[e], 16);
                if (half == 0) ssum[((unit * groups + grp) * a.hc + hh) * kD + 8 * i + e] = __fadd_rn(acc[e], odd) * ks;
            }
        grp = grp1;
        hh = hh1;
    }
    grid_go();
    if (!mean || id < 0) return;
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

// Groups of tokens, counted once for every four key and every eight query heads, from which a warp has two key heads, whose
// angles it reads once from memory: 30,000 tokens of 24 heads 208 us (204 since), with one 233, with four 219; 6,000 70, 66, 77.
constexpr long long kTwoHeads = 8192;

template <typename T, int HC, int PB, bool kFew> cudaError_t launch_append8(AppendArgs &a, cudaStream_t s) {
    const bool all = a.rot == kD && !a.pos;
    const auto kernel = a.inter ? (all ? k_paged8_append<T, true, true, HC, PB, kFew>
                                       : k_paged8_append<T, true, false, HC, PB, kFew>)
                                : (all ? k_paged8_append<T, false, true, HC, PB, kFew>
                                       : k_paged8_append<T, false, false, HC, PB, kFew>);
    const int groups = a.p.page / kGroup;
    a.team = std::min(team_of(a), 8);
    const int warps = a.team > 4 ? a.team : 4, per_cta = warps / a.team;
    const int at_once = 2 * HC * (a.single ? a.team : 1);  // query heads per chunk
    a.kv_chunks = (a.p.Hkv + a.hc - 1) / a.hc;
    a.chunks = a.kv_chunks + (a.q ? (a.p.Hq + at_once - 1) / at_once : 0);
    const long long ctas = (a.units + per_cta - 1) / per_cta * a.chunks;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)warps * 2 * kRawBytes + (a.mean ? sizeof(float) * per_cta * groups * a.hc * kD : 0);
    const cudaError_t e = ensure_smem_limit((const void *)kernel, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_paged(kernel, dim3((unsigned)ctas), 32 * warps, smem, 1, a, s);
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
// values.
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
    const long long page_at = (long long)max(id, 0) * p.page_stride + slot * p.tok_stride;
    if constexpr (KV == 8) {  // 16 dims per lane: the keys and the values of two heads at once
        const int d = 16 * (lane & 7), values = half, odd = (lane >> 3) & 1;
        const unsigned char *from = static_cast<const unsigned char *>(values ? a.vc : a.kc) + page_at + d;
        const float *scale = (values ? a.vs : a.ks) + (long long)max(id, 0) * p.Hkv * (p.page / kGroup) + slot / kGroup;
        T *to = static_cast<T *>(values ? a.v : a.k) + (long long)t * p.Hkv * kD + d;
#pragma unroll 4
        for (int h = h0 + odd; h < h1; h += 2) {
            uint4 w = make_uint4(0, 0, 0, 0);
            float by = 0.f;
            if (id >= 0) {
                w = *reinterpret_cast<const uint4 *>(from + h * p.head_stride);
                by = scale[(long long)h * (p.page / kGroup)];
            }
            float y[8];
            uint4 *out = reinterpret_cast<uint4 *>(to + (long long)h * kD);
            floats_of(make_uint2(w.x, w.y), by, y);
            out[0] = make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
            floats_of(make_uint2(w.z, w.w), by, y);
            out[1] = make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
        }
    } else {  // 8 dims per lane: a head's key and value at once
        const T *from = static_cast<const T *>(half ? a.vc : a.kc) + page_at + 8 * i;
        T *to = static_cast<T *>(half ? a.v : a.k) + (long long)t * p.Hkv * kD + 8 * i;
#pragma unroll 4
        for (int h = h0; h < h1; ++h)
            *reinterpret_cast<uint4 *>(to + (long long)h * kD) =
                id >= 0 ? *reinterpret_cast<const uint4 *>(from + h * p.head_stride) : make_uint4(0, 0, 0, 0);
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
    a.single = !cu_seqlens;
    a.hc = full > kTwoHeads ? 2 : 1;
    // Loops unrolled four deep, and eight query heads per warp, where pages are short or the tokens many; rolled ones, with two
    // heads and four rows, for units of many groups, whose warps are many as it is (us, unrolled / rolled): 1,000 tokens of 8
    // key heads in 64-token pages 10.0 / 10.5, 3,000 16.0 / 19.2, 8 x 1,000 of 2 16.5 / 20.8; 13 x 190 of 3 in 128-token pages
    // 13.7 / 12.2, 4 x 500 of 24 in 256-token ones 26.6 / 22.7, 2 x 3,000 66.5 / 63.5.
    const bool deep = a.p.page <= 64 || full > kTwoHeads;
    cudaError_t e;
    if (a.single)
        e = bf ? launch_append8<__nv_bfloat16, 2, 1, true>(a, s) : launch_append8<__half, 2, 1, true>(a, s);
    else if (deep)
        e = bf ? launch_append8<__nv_bfloat16, 4, 1, false>(a, s) : launch_append8<__half, 4, 1, false>(a, s);
    else
        e = bf ? launch_append8<__nv_bfloat16, 1, 2, true>(a, s) : launch_append8<__half, 1, 2, true>(a, s);
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
