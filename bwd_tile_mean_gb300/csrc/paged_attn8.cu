// paged_attn8.cu -- vsa_paged8_attn and the 8-bit side of
// vsa_paged_attn_weigh. The kernels: paged_attn.cuh.
#include "paged_attn.cuh"

namespace vsa {

namespace {
template <typename T> vsa_status launch8(const AttnArgs &a, bool weigh, cudaStream_t s) {
    if (a.rows <= 8) return weigh ? launch_attn<T, 1, true>(a, s) : launch_attn<T, 1, false>(a, s);
    return weigh ? launch_attn<T, 2, true>(a, s) : launch_attn<T, 2, false>(a, s);
}
}  // namespace

vsa_status attn8(const AttnCall &c, cudaStream_t s) {
    AttnArgs a{};
    const vsa_status st = attn_args(c, true, &a);
    if (st != VSA_OK) return st;
    return a.p.dtype == T_BF16 ? launch8<__nv_bfloat16>(a, c.weigh, s) : launch8<__half>(a, c.weigh, s);
}

}  // namespace vsa

extern "C" vsa_status vsa_paged8_attn(const vsa_paged_desc *desc, const void *q, int64_t q_stride, const void *k_cache,
                                      const void *v_cache, const float *k_scale, const float *v_scale,
                                      const int32_t *page_idx, const int32_t *page_cnt, int idx_cap, void *out, float *lse,
                                      void *workspace, size_t workspace_bytes, vsa_stream_t stream) {
    return vsa::attn8({desc, q, q_stride, k_cache, v_cache, k_scale, v_scale, page_idx, page_cnt, idx_cap, out, lse,
                       workspace, workspace_bytes, false},
                      reinterpret_cast<cudaStream_t>(stream));
}
