// rope.cu -- rotary positions with several axes (vsa_rope_apply, its inverse
// for gradients, and vsa_rope_table): the pairs of a head's dims are divided
// among the axes of a token's position (frame, row, column), pair i of a
// token at position p turns by the angle p[axis(i)] * freq(i).
//
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s;  gradients: the same with -s
//
// Angles: a frequency is kept as a 64-bit fraction of a turn per step, so the
// product with a 32-bit position, modulo 2^64, is the angle's fraction of a
// turn, exact to position * 2^-65 turns however far the position lies; in
// fp32 a position of 100,000 loses 0.004 of a radian. Its upper 32 bits,
// less the quarter turns in them, go to sincospif.
#include <algorithm>
#include <cmath>

#include "paged.cuh"

namespace vsa {
namespace {

struct RopeArgs {
    vsa_rope r;
    int heads0, heads;            // heads of the first tensor, of both
    const void *x[2];
    void *y[2];
    long long xb[2], xt[2], xh[2], yb[2], yt[2], yh[2];
    const int *pos;
    long long pb, pt;
    int S, inverse;
    int chunk, chunks;            // heads per unit, units per token
    long long units;
};

// cos and sin of a fraction of a turn: the quarter turns apart, the rest
// within an eighth of a turn.
__device__ __forceinline__ float2 cos_sin(uint64_t turn) {
    const uint32_t t = (uint32_t)((turn + 0x80000000ull) >> 32);
    const uint32_t q = (t + 0x20000000u) >> 30;
    float c, s;
    sincospif((float)(int32_t)(t - (q << 30)) * 0x1p-31f, &s, &c);
    const float a = q & 1 ? s : c, b = q & 1 ? c : s;
    return make_float2(q == 1 || q == 2 ? -a : a, q & 2 ? -b : b);
}

constexpr int kRopeWarps = 8;
constexpr int kRopeDeep = 4;  // rows per half warp in flight

// A unit is a token and a chunk of its heads (of both tensors, one after the
// other); a warp has one unit at a time, half a warp a head's row: 16 bytes = 8
// dims per lane. Lane l computes the angles of pairs 2 l and 2 l + 1, once for
// all heads of the unit, and every lane gathers those of its own dims. Bound by
// HBM: 76,800 tokens of 40 + 40 heads (3.15 GB) 476 us = 6.6 TB/s, 97% of the
// measured copy rate; 75,600 of 24 + 24 head-major (1.86 GB) 286 us, 96%. 3, 4,
// 6, 8 rows per half warp in flight took 519, 476, 525, 497 us for the former;
// half a warp per token, for tokens side by side, 306 for the latter (299 then).
// kPerSm: CTAs per SM. Tokens whose heads lie side by side go best with three
// (476 us, with four 499), heads whose tokens do with four where pairs are
// interleaved (75,600 tokens of 24 + 24 heads 286, with three 298; 20,000 86, 86;
// 5,000 30, 30). The half style, whose angles take twice the registers, spills
// with four: 325, with three 320; 97, 91; 35, 32.
template <typename T, bool kInter, int kPerSm>
__global__ void __launch_bounds__(kRopeWarps * 32, kPerSm) k_rope(const __grid_constant__ RopeArgs a) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, half = lane >> 4, i = lane & 15;
    const int pairs = a.r.rot_dim >> 1;
    uint64_t turn[2];
    int axis[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const bool on = 2 * lane + e < pairs;
        turn[e] = on ? a.r.turn[2 * lane + e] : 0;
        axis[e] = on ? a.r.axis[2 * lane + e] : 0;
    }
    const int hop = a.r.rot_dim >> 4;  // half style: lanes from a dim to the other of its pair
    const bool on = 8 * i < a.r.rot_dim, lower = i < hop;
    const int peer = (threadIdx.x & 16) | (on ? (lower ? i + hop : i - hop) : i);
    grid_wait();
    for (long long u = (long long)blockIdx.x * kRopeWarps + wid; u < a.units; u += (long long)gridDim.x * kRopeWarps) {
        const long long tok = u / a.chunks;
        const int h0 = (int)(u - tok * a.chunks) * a.chunk, h1 = min(h0 + a.chunk, a.heads);
        const int b = (int)(tok / a.S), s = (int)(tok - (long long)b * a.S);
        const int *pos = a.pos + b * a.pb + s * a.pt;
        float2 mine[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mine[e] = cos_sin((uint64_t)(int64_t)pos[axis[e]] * turn[e]);
            if (a.inverse) mine[e].y = -mine[e].y;
        }
        constexpr int kN = kInter ? 4 : 8;  // angles of a lane's dims
        float c[kN], sn[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            const int from = kInter ? 2 * i + (e >> 1) : 4 * (lower ? i : i - hop) + (e >> 1);
            c[e] = __shfl_sync(0xffffffffu, e & 1 ? mine[1].x : mine[0].x, from & 31);
            sn[e] = __shfl_sync(0xffffffffu, e & 1 ? mine[1].y : mine[0].y, from & 31);
            if (!kInter && lower) sn[e] = -sn[e];
        }
        for (int h = h0 + half; h - half < h1; h += 2 * kRopeDeep) {
            uint4 x[kRopeDeep];
            long long at[kRopeDeep];
#pragma unroll
            for (int d = 0; d < kRopeDeep; ++d) {
                const int hh = h + 2 * d, k = hh >= a.heads0, hk = hh - (k ? a.heads0 : 0);
                at[d] = b * a.yb[k] + s * a.yt[k] + hk * a.yh[k] + 8 * i;
                x[d] = make_uint4(0, 0, 0, 0);
                if (hh < h1)
                    x[d] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x[k]) + b * a.xb[k] + s * a.xt[k] +
                                                            hk * a.xh[k] + 8 * i);
            }
#pragma unroll
            for (int d = 0; d < kRopeDeep; ++d) {
                uint32_t r[4] = {x[d].x, x[d].y, x[d].z, x[d].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = unpack2<T>(r[j]);
                    if constexpr (kInter) {
                        const uint32_t y = pack2<T>(__fsub_rn(__fmul_rn(v.x, c[j]), __fmul_rn(v.y, sn[j])),
                                                    __fadd_rn(__fmul_rn(v.y, c[j]), __fmul_rn(v.x, sn[j])));
                        r[j] = on ? y : r[j];
                    } else {
                        const float2 w = unpack2<T>(__shfl_sync(0xffffffffu, r[j], peer));
                        // lower dims: x1 c + x2 (-s), the same bits as x1 c - x2 s
                        const uint32_t y = pack2<T>(__fadd_rn(__fmul_rn(v.x, c[2 * j]), __fmul_rn(w.x, sn[2 * j])),
                                                    __fadd_rn(__fmul_rn(v.y, c[2 * j + 1]), __fmul_rn(w.y, sn[2 * j + 1])));
                        r[j] = on ? y : r[j];
                    }
                }
                const int hh = h + 2 * d;
                if (hh < h1)
                    *reinterpret_cast<uint4 *>(static_cast<T *>(a.y[hh >= a.heads0]) + at[d]) =
                        make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
    }
    grid_go();
}

// Bound by its instructions, a 64-bit division among them: 100, 6,000, 76,800
// tokens of 64 pairs 1.9, 4.2, 20.4 us, where the bytes of the last take 5.8.
struct TableArgs {
    vsa_rope r;
    const int *pos;
    long long pt, n;  // angles in all
    float *cos, *sin;
};
__global__ void __launch_bounds__(256) k_rope_table(const __grid_constant__ TableArgs a) {
    __shared__ uint64_t s_turn[64];
    __shared__ int s_axis[64];
    const int pairs = a.r.rot_dim >> 1;
    if (threadIdx.x < pairs) {
        s_turn[threadIdx.x] = a.r.turn[threadIdx.x];
        s_axis[threadIdx.x] = a.r.axis[threadIdx.x];
    }
    __syncthreads();
    grid_wait();
    for (long long at = (long long)blockIdx.x * 256 + threadIdx.x; at < a.n; at += (long long)gridDim.x * 256) {
        const long long t = at / pairs;
        const int i = (int)(at - t * pairs);
        const float2 cs = cos_sin((uint64_t)(int64_t)a.pos[t * a.pt + s_axis[i]] * s_turn[i]);
        a.cos[at] = cs.x;
        a.sin[at] = cs.y;
    }
    grid_go();
}

vsa_status check_rope(const vsa_rope *r) {
    if (!r) return VSA_ERR_NULL;
    if (r->n_axes < 1 || r->n_axes > VSA_ROPE_AXES) return VSA_ERR_SHAPE;
    if (r->rot_dim < 16 || r->rot_dim > kD || r->rot_dim % 16 != 0) return VSA_ERR_UNSUPPORTED;
    for (int i = 0; i < r->rot_dim / 2; ++i)
        if (r->axis[i] >= r->n_axes) return VSA_ERR_SHAPE;
    return VSA_OK;
}

// frac(f / (2 pi)) as a 64-bit fraction, rounded. f = m 2^e with a 53-bit m;
// 1 / (2 pi) to 192 bits below the point (its first ones: 2^-3).
uint64_t turn_of(double f) {
    if (f == 0.0) return 0;
    static const uint32_t inv[6] = {0x28be60dbu, 0x9391054au, 0x7f09d5f4u, 0x7d4d3770u, 0x36d8a566u, 0x4f10e410u};
    int e;
    const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(f), &e), 53);
    e -= 53;
    // product of m and the fraction: 8 words of 32 bits, w[0] the highest; the point lies behind w[1]
    uint32_t w[8] = {};
    for (int part = 0; part < 2; ++part) {  // low and high word of m
        const uint64_t mp = part ? m >> 32 : m & 0xffffffffu;
        uint64_t carry = 0;
        for (int k = 5; k >= 0; --k) {
            const int at = k + 2 - part;
            const uint64_t x = mp * inv[k] + w[at] + carry;
            w[at] = (uint32_t)x;
            carry = x >> 32;
        }
        for (int at = 1 - part; at >= 0 && carry; --at) {
            const uint64_t x = w[at] + carry;
            w[at] = (uint32_t)x;
            carry = x >> 32;
        }
    }
    // the bits 1 .. 64 behind the point of the product times 2^e, and one more to round by
    auto bit = [&](int behind) -> uint64_t {  // of the product: bit `behind` behind the point (1 is a half)
        const int at = 64 + behind - 1;
        return at < 0 || at >= 256 ? 0 : (w[at >> 5] >> (31 - (at & 31))) & 1u;
    };
    uint64_t t = 0;
    for (int i = 1; i <= 64; ++i) t = (t << 1) | bit(i + e);
    t += bit(65 + e);
    return f < 0 ? 0 - t : t;
}

}  // namespace
}  // namespace vsa

using namespace vsa;

extern "C" vsa_status vsa_rope_init(vsa_rope *rope, int n_axes, int rot_dim, int interleaved, const int32_t *axis,
                                    const double *freq) {
    if (!rope || !axis || !freq) return VSA_ERR_NULL;
    vsa_rope r{};
    r.n_axes = n_axes;
    r.rot_dim = rot_dim;
    r.interleaved = interleaved != 0;
    if (rot_dim < 16 || rot_dim > kD || rot_dim % 16 != 0) return VSA_ERR_UNSUPPORTED;
    for (int i = 0; i < rot_dim / 2; ++i) {
        if (axis[i] < 0 || axis[i] >= n_axes || !(std::fabs(freq[i]) <= 1024.0)) return VSA_ERR_SHAPE;
        r.axis[i] = (uint8_t)axis[i];
        r.turn[i] = turn_of(freq[i]);
    }
    const vsa_status st = check_rope(&r);
    if (st == VSA_OK) *rope = r;
    return st;
}

extern "C" vsa_status vsa_rope_apply(const vsa_rope *rope, int dtype, int B, int S, int D, const vsa_rope_tensor *t, int n,
                                     const int32_t *positions, int64_t pos_batch, int64_t pos_token, int inverse,
                                     vsa_stream_t stream) {
    const vsa_status st = check_rope(rope);
    if (st != VSA_OK) return st;
    if (dtype != VSA_DTYPE_BF16 && dtype != VSA_DTYPE_FP16) return VSA_ERR_DTYPE;
    if (D != kD) return VSA_ERR_UNSUPPORTED;
    if (B < 0 || S < 0 || n < 1 || n > 2) return VSA_ERR_SHAPE;
    if (!t) return VSA_ERR_NULL;
    const bool none = B == 0 || S == 0;
    RopeArgs a{};
    long long heads = 0;
    for (int k = 0; k < n; ++k) {
        if (t[k].heads < 1) return VSA_ERR_SHAPE;
        const int64_t strides[6] = {t[k].x_batch, t[k].x_token, t[k].x_head, t[k].y_batch, t[k].y_token, t[k].y_head};
        for (const int64_t x : strides)
            if (x < 0 || x % 8 != 0) return VSA_ERR_SHAPE;
        if (!none && (!t[k].x || !t[k].y)) return VSA_ERR_NULL;
        if (!aligned16(t[k].x) || !aligned16(t[k].y)) return VSA_ERR_LAYOUT;
        a.x[k] = t[k].x;
        a.y[k] = t[k].y;
        a.xb[k] = t[k].x_batch, a.xt[k] = t[k].x_token, a.xh[k] = t[k].x_head;
        a.yb[k] = t[k].y_batch, a.yt[k] = t[k].y_token, a.yh[k] = t[k].y_head;
        heads += t[k].heads;
    }
    if (heads > 0x7fffffffLL || (long long)B * S > 0x7fffffffLL) return VSA_ERR_UNSUPPORTED;
    if (pos_batch < 0 || pos_token < 0) return VSA_ERR_SHAPE;
    if ((uintptr_t)positions & 3u) return VSA_ERR_LAYOUT;
    if (none) return VSA_OK;
    if (!positions) return VSA_ERR_NULL;
    a.r = *rope;
    a.heads0 = t[0].heads;
    a.heads = (int)heads;
    a.pos = positions;
    a.pb = pos_batch;
    a.pt = pos_token;
    a.S = S;
    a.inverse = inverse != 0;
    const long long tokens = (long long)B * S, places = 152 * 64;
    // all heads of a token in one unit, or as many units as fill the GPU's warps (5,757 tokens of 15 heads 12.8 us, in three
    // units each 17.4: each computes the angles)
    long long chunks = std::min((heads + 2 * kRopeDeep - 1) / (2 * kRopeDeep), std::max(1LL, places / tokens));
    a.chunk = (int)((heads + chunks - 1) / chunks);
    a.chunk = (a.chunk + 1) & ~1;
    a.chunks = (int)((heads + a.chunk - 1) / a.chunk);
    a.units = tokens * a.chunks;
    // twice the CTAs that fit: with three of them 3, 4, 5, 6, 8, 32 per SM took 475, 548, 498, 476, 486, 487 us
    const bool four = a.r.interleaved && S > 1 && t[0].x_token < t[0].x_head;
    const unsigned grid = (unsigned)std::min((a.units + kRopeWarps - 1) / kRopeWarps, four ? 152LL * 8 : 152LL * 6);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    prof_begin("rope", s);
    const bool bf = dtype == VSA_DTYPE_BF16;
    const auto kernel =
        four ? (bf ? k_rope<__nv_bfloat16, true, 4> : k_rope<__half, true, 4>)
             : (a.r.interleaved ? (bf ? k_rope<__nv_bfloat16, true, 3> : k_rope<__half, true, 3>)
                                : (bf ? k_rope<__nv_bfloat16, false, 3> : k_rope<__half, false, 3>));
    const cudaError_t e = launch_paged(kernel, dim3(grid), kRopeWarps * 32, 0, 1, a, s);
    prof_end(s);
    return status_from_cuda(e);
}

extern "C" vsa_status vsa_rope_table(const vsa_rope *rope, int T, const int32_t *positions, int64_t pos_token, float *cos,
                                     float *sin, vsa_stream_t stream) {
    const vsa_status st = check_rope(rope);
    if (st != VSA_OK) return st;
    if (T < 0 || pos_token < 0) return VSA_ERR_SHAPE;
    if (T == 0) return VSA_OK;
    if (!positions || !cos || !sin) return VSA_ERR_NULL;
    if ((uintptr_t)positions & 3u || !aligned16(cos) || !aligned16(sin)) return VSA_ERR_LAYOUT;
    TableArgs a{*rope, positions, pos_token, (long long)T * (rope->rot_dim / 2), cos, sin};
    const unsigned grid = (unsigned)std::min((a.n + 255) / 256, 152LL * 8);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    prof_begin("rope_table", s);
    const cudaError_t e = launch_paged(k_rope_table, dim3(grid), 256, 0, 1, a, s);
    prof_end(s);
    return status_from_cuda(e);
}
