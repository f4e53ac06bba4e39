// paged_attn.cu -- vsa_paged_attn, the 16-bit side of vsa_paged_attn_weigh,
// and the workspaces. The kernels: paged_attn.cuh.
#include "paged_attn.cuh"

namespace vsa {

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
    w.ml = take(sizeof(float4) * 2 * kCtas * kWarps * rows);
    w.o = take(sizeof(float) * 2 * kCtas * kWarps * rows * kD);
    w.stat = take(sizeof(float2) * p.B * (size_t)p.Hq);
    w.total = at;
    return w;
}

size_t weigh_bytes(const Paged &p) {
    const size_t rows = rows_of(p.G), rc = (p.G + rows - 1) / rows;
    return paged_ws(p).total + sizeof(float2) * p.B * (size_t)p.Hkv * rc * p.max_pages * (p.page / kBlk) * rows;
}

vsa_status attn16(const AttnCall &c, cudaStream_t s) {
    AttnArgs a{};
    const vsa_status st = attn_args(c, false, &a);
    if (st != VSA_OK) return st;
    if (c.weigh) return a.p.dtype == T_BF16 ? launch_attn<__nv_bfloat16, 0, true>(a, s) : launch_attn<__half, 0, true>(a, s);
    return a.p.dtype == T_BF16 ? launch_attn<__nv_bfloat16, 0, false>(a, s) : launch_attn<__half, 0, false>(a, s);
}

}  // namespace vsa

extern "C" size_t vsa_paged_workspace_size(const vsa_paged_desc *desc) {
    vsa::Paged p;
    if (vsa::to_paged(desc, &p, false) != VSA_OK) return 0;
    return vsa::paged_ws(p).total;
}

extern "C" size_t vsa_paged_weigh_workspace_size(const vsa_paged_desc *desc) {
    vsa::Paged p;
    if (vsa::to_paged(desc, &p, false) != VSA_OK) return 0;
    return vsa::weigh_bytes(p);
}

extern "C" vsa_status vsa_paged_attn(const vsa_paged_desc *desc, const void *q, int64_t q_stride,
                                     const void *k_cache, const void *v_cache, const int32_t *page_idx,
                                     const int32_t *page_cnt, int idx_cap, void *out, float *lse, void *workspace,
                                     size_t workspace_bytes, vsa_stream_t stream) {
    return vsa::attn16({desc, q, q_stride, k_cache, v_cache, nullptr, nullptr, page_idx, page_cnt, idx_cap, out, lse,
                        workspace, workspace_bytes, false},
                       reinterpret_cast<cudaStream_t>(stream));
}
