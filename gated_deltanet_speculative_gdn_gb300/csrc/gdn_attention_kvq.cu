// gdn_attention_kvq.cu - attention over the paged cache held in 4 bits: the kernel of
// gdn_attention.cuh with keys and values that are converted on their way to the tensor
// cores (its mathematics, work and mapping are in gdn_attention.cu).
//
// Rounding.  Codes times scales have 6 significant bits and are multiples of 2^-10 up to
// 2688, so fp16 holds them exactly: both products run in fp16 whatever q's type, p rounded
// as for an fp16 cache.  fp16 q rows go in as they are, bf16 rows scaled by a power of two
// by row.  The units are factors of the scores and of the result.
//
// Mapping.  Beside the rows' warps (4, or 8 for d <= 128) and the two that issue products
// stand d / 32 warps that take the place of TMA: every thread copies the codes and scales of
// its own 64 elements of a tile kAhead tiles early (cp.async), converts them (one cvt and one
// product for two elements) and writes them to the ring of tiles as fp16 in the 128-byte
// swizzle.
#include "gdn_attention.cuh"

namespace {

template <typename T, int D>
__global__ void __launch_bounds__(att::Cfg<D, true>::kThreads, 1) kvq_attention_kernel(const att::Args a) {
    attention_body<T, D, true>(nullptr, nullptr, a);
}

template <typename T, int D>
int launch(const gdn_attn_dims *dims, att::Args a, void *workspace, int ctas, cudaStream_t st) {
    using C = att::Cfg<D, true>;
    a.meta = static_cast<int4 *>(workspace);
    a.parts = reinterpret_cast<float *>(a.meta + 2 * ctas);
    a.stall_ns = gdn::take_attention_stall(&a.stall_role);
    auto k = kvq_attention_kernel<T, D>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem)) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    if (gdn::launch_pdl(k, dim3(unsigned(ctas)), dim3(C::kThreads), C::kSmem, st, a) != cudaSuccess) return GDN_ERR_LAUNCH;
    return launch_join<T, D, true>(dims, a, ctas, st);
}

template <typename T>
int launch_d(const gdn_attn_dims *dims, const att::Args &a, void *workspace, int ctas, cudaStream_t st) {
    switch (dims->d_head) {
        case 64: return launch<T, 64>(dims, a, workspace, ctas, st);
        case 128: return launch<T, 128>(dims, a, workspace, ctas, st);
        default: return launch<T, 256>(dims, a, workspace, ctas, st);
    }
}

}  // namespace

extern "C" size_t gdn_attention_kvq_workspace_bytes(const gdn_attn_dims *dims) {
    if (gdn::check_kv4_dims(dims) != GDN_OK) return 0;
    const int ctas = gdn::sm_count_current();
    return workspace_bytes(dims, ctas > 0 ? ctas : 1);
}

extern "C" int gdn_paged_attention_kvq(const gdn_attn_dims *dims, const void *q, int64_t q_stride, const void *k_pool,
                                       const void *v_pool, float k_unit, float v_unit, const int32_t *page_table,
                                       const int32_t *ctx_len, const int32_t *node_off, const int32_t *parents, float scale,
                                       void *o, void *workspace, int64_t workspace_size, int32_t *status, void *stream) {
    int rc = gdn::check_kv4_dims(dims);
    if (rc) return rc;
    if (!gdn::good_unit(k_unit) || !gdn::good_unit(v_unit)) return GDN_ERR_ARG;
    bool empty = false;
    rc = check_attention(dims, q, q_stride, k_pool, v_pool, gdn::kv4_pool_bytes(dims), page_table, ctx_len, node_off, parents, scale, o,
                         workspace, workspace_size, gdn_attention_kvq_workspace_bytes(dims), status, &empty);
    if (rc || empty) return rc;
    const int ctas = gdn::sm_count_current();
    if (ctas < 1) return GDN_ERR_LAUNCH;
    const int64_t S = dims->n_seqs, N = dims->n_tokens, Hq = dims->h_q;
    const int G = int(Hq / dims->h_kv);
    att::Args a{q, q_stride, k_pool, v_pool, gdn::paged_layout(dims, page_table), ctx_len, node_off, parents,
                scale * k_unit * 1.4426950408889634f, v_unit, o, status, nullptr, nullptr, int(S), int(N), dims->max_seq_tokens,
                int(Hq), dims->h_kv, G, att::kRows / G, 0, 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dims->dtype == GDN_BF16 ? launch_d<__nv_bfloat16>(dims, a, workspace, ctas, st)
                                   : launch_d<__half>(dims, a, workspace, ctas, st);
}
