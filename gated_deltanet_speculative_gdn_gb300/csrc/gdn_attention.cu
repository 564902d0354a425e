// gdn_attention.cu - attention of a chunk of new tokens over a paged cache: the
// full-attention layers of a speculative round (token trees), of a prompt's chunk
// and of plain decode, in one kernel.
//
// Mathematics.  One pass over the positions with a running reference m and sum l:
//     p_x = 2^(c s_x - m),  l += p_x,  O += p_x v_x,   c = scale log2(e)
// where m is the largest c s of the first tile that the row sees, or of the tile for
// which it was last moved, less kLift.  It is moved (l and O scaled by 2^(m - m')) only
// when p would pass 2^kMoveAt: until then p is in the type's range, and a scale costs
// no precision in a floating type.  With one warpgroup (D = 256) the exponentials are
// formed without a look at the maximum, which would stand before all of them in the
// longest chain of the kernel; a tile whose p sum to more than kMoveAtSum (so one p
// alone may reach that) has its m moved and its p formed again.  (With two, keeping the
// scores for that costs registers that spill: 270 -> 330 us for chunks of up to 701
// tokens at D = 128.)  Parts of a row's positions are joined by the same rule:
// o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
//
// Rounding.  The products run on the tensor cores with 16-bit operands and fp32
// accumulators, so p is rounded to the cache's type before P V: a relative half
// step of that type, as the result's own rounding; l sums the unrounded p.  bf16 has
// fp32's range.  fp16 has steps of 2^-24 below 2^-14, so its range is used from the
// top: the largest p of a row is 2^8 at least (kLift) and 2^15.9 at most, weights down
// to 2^-22 of the largest keep their relative half step, and smaller ones are off by
// 2^-33 of it at most.  (16,384 positions that stand 18 nats below one other with a
// hundredth of their value: 9 to 17 times the roundings' bound with m at the maximum
// itself, 0.3 to 0.4 of it so.  Mixed chunks in fp16 took 262 us and take 265, trees in fp16 and
// bf16 the same to 2 % with flat scores and with peaked ones.)
//
// Work.  The h_q / h_kv heads that share a key/value head are rows of one tile:
// row r is (token i0 + r / G, head r % G), 128 / G tokens a tile, so keys and
// values are read once for all of them.  An item is (sequence, key/value head, row
// tile); its positions come in tiles of TK.  All items in a row, each its tiles and
// a few tiles' worth for its beginning and end, are cut into equal shares, one per
// CTA (one CTA per SM): lengths as ragged as they come keep every SM busy to the end,
// one sequence alone spreads over the GPU, and a CTA has at most one item that began
// before it and one that ends after it.  Those parts go to the workspace and a second
// kernel joins them in CTA order, so results do not depend on timing.
//
// Mapping (GB300).  Tensor memory holds O (D columns, fp32), Q (D / 2 columns, the
// A operand of Q K^T: nothing of it is read again from shared memory, which leaves
// all of that to keys and values), one score tile per warpgroup (64 columns) and two
// of P (32 columns, the A operand of P V), so that the next scores need not wait for
// the product.  Shared memory is a ring of 192 KB of key and value tiles, filled by
// TMA page by page in the 128-byte swizzle: keys as they lie are the K-major B
// operand, values as they lie the MN-major one.
//   rows    four warps, row r = 32 w + lane = tensor-memory lane: Q in, scores -> P,
//           moves of m, results out.  For D <= 128 the softmax is longer than the
//           products: two warpgroups take alternate tiles, each with an O, m and l of
//           its own, joined at the end of a segment.
//   TMA     K_0 K_1 V_0 K_2 V_1 ...  A box costs ~90 cycles whatever it holds, so a
//           page (from 16 tokens on) is one box, and the products take a tile page by
//           page.  As a box per page and 64 columns, pages of 16 took 1165 us and
//           pages of 64 688 us for the chunk of 4096 over 12288 positions.
//   mma     two warps: S_{i+1} = Q K_{i+1}^T runs while P_i is formed (one warp's waits
//           for one product kept it from the other: 745 -> 724 us, and 592 with P's own place)
//   clean   values of tiles in which some rows do not see some positions: what no row
//           sees (the rest of a page) is set to 0, and elements that are not finite
//           are set to 0 and remembered, since 0 * NaN in P V would reach rows that
//           do not see them; rows that do get them back at the end
//
// Measured (16/2 heads of 256, bf16): 64 single tokens over up to 16,384 positions 184-189 us, 6.3-6.4 TB/s, HBM;
// 64 trees of 16 nodes over up to 8,192 119-122 us, 5.0-5.1 TB/s, HBM and the parts' way through memory; 4,096 tokens over
// 12,288 positions 533-616 us, 1.56-1.8 PFLOP/s, tensor cores under the power cap; one token over 777 positions
// 14 us, latency.
//
// Every mbarrier completes once per use, so a counter gives every wait's phase; a
// wait is only ever for the next completion that the waiter has not seen.
#include <algorithm>
#include <atomic>

#include "gdn_attention.cuh"

namespace {

template <typename T, int D>
__global__ void __launch_bounds__(att::Cfg<D>::kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                           const att::Args a) {
    attention_body<T, D, false>(&kmap, &vmap, a);
}

// A paged pool viewed as [page][head][d / 64][token][64], boxes of [chunks][rows tokens][64] of one head and
// page in the 128-byte swizzle; GDN_OK or GDN_ERR_TMA.
int encode_kv_pages(CUtensorMap *map, const void *pool, const gdn_attn_dims *d, uint32_t rows, uint32_t chunks) {
    static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!enc) return GDN_ERR_TMA;
    const cuuint64_t gdim[5] = {64, cuuint64_t(d->page_size), cuuint64_t(d->d_head / 64), cuuint64_t(d->h_kv),
                                cuuint64_t(d->n_pages)};
    const cuuint64_t gstride[4] = {cuuint64_t(d->token_stride) * 2, 128, cuuint64_t(d->head_stride) * 2,
                                   cuuint64_t(d->page_stride) * 2};
    const cuuint32_t box[5] = {64, rows, chunks, 1, 1}, estride[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, const_cast<void *>(pool), gdim, gstride, box, estride,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GDN_OK : GDN_ERR_TMA;
}

template <typename T, int D>
int launch(const gdn_attn_dims *dims, att::Args a, void *workspace, int ctas, cudaStream_t st) {
    using C = att::Cfg<D>;
    CUtensorMap kmap, vmap;
    const int ps = dims->page_size;
    const uint32_t rows = uint32_t(ps < att::TK ? ps : att::TK);
    int rc;
    const uint32_t chunks = ps >= 16 ? C::kChunks : 1;
    if ((rc = encode_kv_pages(&kmap, a.k_pool, dims, rows, chunks)) ||
        (rc = encode_kv_pages(&vmap, a.v_pool, dims, rows, chunks)))
        return rc;
    a.meta = static_cast<int4 *>(workspace);
    a.parts = reinterpret_cast<float *>(a.meta + 2 * ctas);
    a.stall_ns = gdn::take_attention_stall(&a.stall_role);
    auto k = paged_attention_kernel<T, D>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem)) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    if (gdn::launch_pdl(k, dim3(unsigned(ctas)), dim3(C::kThreads), C::kSmem, st, kmap, vmap, a) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    return launch_join<T, D, false>(dims, a, ctas, st);
}

template <typename T>
int launch_d(const gdn_attn_dims *dims, const att::Args &a, void *workspace, int ctas, cudaStream_t st) {
    switch (dims->d_head) {
        case 64: return launch<T, 64>(dims, a, workspace, ctas, st);
        case 128: return launch<T, 128>(dims, a, workspace, ctas, st);
        default: return launch<T, 256>(dims, a, workspace, ctas, st);
    }
}

std::atomic<uint64_t> g_stall{0};  // the pending test stall: role in the top byte, ns below

}  // namespace

uint64_t gdn::take_attention_stall(int *role) {
    const uint64_t stall = g_stall.exchange(0);
    *role = int(stall >> 56);
    return stall & ((uint64_t(1) << 56) - 1);
}

extern "C" size_t gdn_attention_workspace_bytes(const gdn_attn_dims *dims) {
    if (gdn::check_attn_dims(dims) != GDN_OK) return 0;
    const int ctas = gdn::sm_count_current();
    return workspace_bytes(dims, ctas > 0 ? ctas : 1);
}

extern "C" int gdn_paged_attention(const gdn_attn_dims *dims, const void *q, int64_t q_stride, const void *k_pool,
                                   const void *v_pool, const int32_t *page_table, const int32_t *ctx_len,
                                   const int32_t *node_off, const int32_t *parents, float scale, void *o, void *workspace,
                                   int64_t workspace_size, int32_t *status, void *stream) {
    int rc = gdn::check_attn_dims(dims);
    if (rc) return rc;
    bool empty = false;
    rc = check_attention(dims, q, q_stride, k_pool, v_pool, gdn::pool_bytes(dims), page_table, ctx_len, node_off, parents, scale, o,
                         workspace, workspace_size, gdn_attention_workspace_bytes(dims), status, &empty);
    if (rc || empty) return rc;
    const int64_t S = dims->n_seqs, N = dims->n_tokens, Hq = dims->h_q;
    const int ctas = gdn::sm_count_current();
    if (ctas < 1) return GDN_ERR_LAUNCH;
    const int G = int(Hq / dims->h_kv);
    att::Args a{q, q_stride, k_pool, v_pool, gdn::paged_layout(dims, page_table), ctx_len, node_off, parents,
                scale * 1.4426950408889634f, 1.f, 0, 1.f, o, status, nullptr, nullptr, int(S), int(N), dims->max_seq_tokens, int(Hq),
                dims->h_kv, G, att::kRows / G, 0, 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dims->dtype == GDN_BF16 ? launch_d<__nv_bfloat16>(dims, a, workspace, ctas, st)
                                   : launch_d<__half>(dims, a, workspace, ctas, st);
}

extern "C" void gdn_test_stall_next_attention(uint64_t wait_ns, int role) {
    if (role < 0 || role > 4) return;
    g_stall.store(std::min<uint64_t>(wait_ns, gdn::kWaitLimitNs) | (uint64_t(role) << 56));
}
