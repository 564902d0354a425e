// gdn_attention.cu - attention of a chunk of new tokens over a paged cache.
//
// First form: a warp per (token, query head), one pass over the positions it
// sees with a running maximum and sum.
#include "gdn_attn.h"

namespace {

struct AttnArgs {
    const void *__restrict__ q;
    int64_t q_stride;
    const void *__restrict__ k_pool, *__restrict__ v_pool;
    gdn::PagedLayout pl;
    const int32_t *__restrict__ ctx_len, *__restrict__ node_off, *__restrict__ parents;
    float scale;
    void *o;
    int32_t *status;
    int S, N, max_tokens, Hq, Hkv;
};

template <typename T, int D>
__global__ void __launch_bounds__(128) paged_attention_kernel(const AttnArgs a) {
    constexpr int E = D / 32;  // elements of a lane
    const unsigned full = 0xffffffffu;
    gdn::grid_dep_launch();
    gdn::grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t wid = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (blockIdx.x == 0) {
        const int err = gdn::check_node_off(a.node_off, a.S, a.N, a.max_tokens, threadIdx.x, 128);
        if (err) gdn::record_status(a.status, err);
    }
    const int n = int(wid / a.Hq), h = int(wid % a.Hq), hk = h / (a.Hq / a.Hkv);
    if (n >= a.N) return;
    const int s = gdn::find_sequence(a.node_off, a.S, n);
    const int n0 = a.node_off[s], i = n - n0, ctx = a.ctx_len[s];
    int err = 0;
    if (i < 0 || i >= a.max_tokens || n >= a.node_off[s + 1]) err = GDN_DEV_BAD_NODE_OFF;
    else if (ctx < 0 || int64_t(ctx) + i >= (int64_t(a.pl.width) << a.pl.shift)) err = GDN_DEV_BAD_LEN;
    unsigned long long line = 0;
    if (!err && a.parents) {
        for (int x = i; x >= 0;) {
            line |= 1ull << x;
            const int p = a.parents[n0 + x];
            if (p >= x || p < -1) { err = GDN_DEV_BAD_PARENT; break; }
            x = p;
        }
    }
    if (err) {
        if (lane == 0) gdn::record_status(a.status, err);
        return;
    }
    float q[E], o[E], m = -INFINITY, l = 0.f;
    const T *qr = static_cast<const T *>(a.q) + n * a.q_stride + int64_t(h) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = float(qr[e]);
        o[e] = 0.f;
    }
    for (int x = 0; x <= ctx + i; ++x) {
        if (x >= ctx && a.parents && !((line >> (x - ctx)) & 1)) continue;
        const int64_t at = gdn::position_offset(a.pl, s, x);
        if (at < 0) {
            if (lane == 0) gdn::record_status(a.status, GDN_DEV_BAD_PAGE);
            return;
        }
        const T *kr = static_cast<const T *>(a.k_pool) + at + int64_t(hk) * a.pl.head_stride + lane * E;
        const T *vr = static_cast<const T *>(a.v_pool) + at + int64_t(hk) * a.pl.head_stride + lane * E;
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) d = fmaf(q[e], float(kr[e]), d);
        d = gdn::warp_sum(d) * a.scale;
        const float mn = fmaxf(m, d);
        const float al = m == -INFINITY ? 0.f : expf(m - mn), p = expf(d - mn);
        l = l * al + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p, float(vr[e]), al == 0.f ? 0.f : o[e] * al);
        m = mn;
    }
    T *orow = static_cast<T *>(a.o) + (int64_t(n) * a.Hq + h) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) orow[e] = T(o[e] / l);
    (void)full;
}

template <typename T>
cudaError_t launch(int d, dim3 grid, cudaStream_t st, const AttnArgs &a) {
    switch (d) {
        case 64: return gdn::launch_pdl(paged_attention_kernel<T, 64>, grid, dim3(128), 0, st, a);
        case 128: return gdn::launch_pdl(paged_attention_kernel<T, 128>, grid, dim3(128), 0, st, a);
        default: return gdn::launch_pdl(paged_attention_kernel<T, 256>, grid, dim3(128), 0, st, a);
    }
}

}  // namespace

extern "C" size_t gdn_attention_workspace_bytes(const gdn_attn_dims *dims) {
    return gdn::check_attn_dims(dims) == GDN_OK ? 16 : 0;
}

extern "C" int gdn_paged_attention(const gdn_attn_dims *dims, const void *q, int64_t q_stride, const void *k_pool,
                                   const void *v_pool, const int32_t *page_table, const int32_t *ctx_len,
                                   const int32_t *node_off, const int32_t *parents, float scale, void *o, void *workspace,
                                   int64_t workspace_bytes, int32_t *status, void *stream) {
    int rc = gdn::check_attn_dims(dims);
    if (rc) return rc;
    if (!status) return GDN_ERR_NULL;
    if (parents && dims->max_seq_tokens > gdn::kMaxSeqNodes) return GDN_ERR_DIMS;
    if (!(scale > 0.0f) || !(scale < 3.0e38f)) return GDN_ERR_ARG;
    const int64_t S = dims->n_seqs, N = dims->n_tokens, Hq = dims->h_q, D = dims->d_head;
    if (S == 0 || N == 0) return GDN_OK;
    if (!q || !k_pool || !v_pool || !page_table || !ctx_len || !node_off || !o || !workspace) return GDN_ERR_NULL;
    const size_t need = gdn_attention_workspace_bytes(dims);
    if (workspace_bytes < 0 || size_t(workspace_bytes) < need) return GDN_ERR_ARG;
    if (q_stride < Hq * D || q_stride % 8) return GDN_ERR_STRIDE;
    if (!gdn::aligned16(q) || !gdn::aligned16(k_pool) || !gdn::aligned16(v_pool) || !gdn::aligned16(o) ||
        !gdn::aligned16(workspace))
        return GDN_ERR_ALIGN;
    const size_t pool = gdn::pool_bytes(dims);
    const gdn::Span outs[] = {{o, size_t(N * Hq * D * 2)}, {workspace, need}};
    const gdn::Span ins[] = {{q, gdn::rows_bytes16(N, q_stride, Hq * D)},
                             {k_pool, pool},
                             {v_pool, pool},
                             {page_table, size_t(S * int64_t(dims->table_width) * 4)},
                             {ctx_len, size_t(S * 4)},
                             {node_off, size_t((S + 1) * 4)},
                             {parents, size_t(N * 4)},
                             {status, 4}};
    if ((rc = gdn::check_alias(outs, 2, ins, 8))) return rc;
    AttnArgs a{q, q_stride, k_pool, v_pool, gdn::paged_layout(dims, page_table), ctx_len, node_off, parents, scale, o,
               status, int(S), int(N), dims->max_seq_tokens, int(Hq), dims->h_kv};
    const dim3 grid(unsigned((N * Hq + 3) / 4));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dims->dtype == GDN_BF16 ? launch<__nv_bfloat16>(int(D), grid, st, a)
                                                  : launch<__half>(int(D), grid, st, a);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
