// paged_attn8.cu -- vsa_paged8_attn and the 8-bit side of
// vsa_paged_attn_weigh. The kernels: paged_attn.cuh.
#include "paged_attn.cuh"

namespace vsa {

vsa_status attn8(const AttnCall &c, cudaStream_t s) {
    AttnArgs a{};
    const vsa_status st = attn_args(c, true, &a);
    if (st != VSA_OK) return st;
    if (c.weigh) return a.p.dtype == T_BF16 ? launch_attn<__nv_bfloat16, 8, true>(a, s) : launch_attn<__half, 8, true>(a, s);
    return a.p.dtype == T_BF16 ? launch_attn<__nv_bfloat16, 8, false>(a, s) : launch_attn<__half, 8, false>(a, s);
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
