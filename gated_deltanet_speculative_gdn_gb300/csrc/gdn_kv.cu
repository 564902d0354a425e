// gdn_kv.cu - commit of the accepted path in the paged cache: the attention
// layers' part of a speculative round's commit (the GDN layers' is gdn_commit.cu),
// all layers in one call.
//
// The new tokens of a round lie at positions ctx + 0, 1, ... in node order; once
// a path p_0 < p_1 < ... < p_{m-1} is accepted its rows move to ctx + 0 .. m - 1.
// As p_j >= j, a row never moves over one that is still to be read when the path
// is taken in order; a thread owns one 16-byte column of one layer's keys or
// values and takes the whole path, so no two threads touch the same bytes.  It
// loads up to 8 rows, then stores them (a store goes to j <= p_j, below every
// row that a later load reads).
//
// Two launches, as gdn_commit: a preflight checks every sequence and writes
// *status, the move writes nothing unless it is zero.  Bound by latency: a
// round's rows are a few MB at most, and the floor is three dependent round trips
// (path, page table, rows).  12 layers of 64 sequences take 4.7 us in a graph.
#include "gdn_attn.h"

namespace {

struct KvArgs {
    const int32_t *__restrict__ accepted, *__restrict__ parents, *__restrict__ node_off, *__restrict__ ctx_len;
    gdn::PagedLayout pl;
    void *k_pool, *v_pool;
    int64_t layer_stride;
    int32_t *new_len;
    int32_t *status;
    int S, N, max_tokens, Hkv, cols;  // cols: 16-byte columns of a token's keys, h_kv * d / 8
    int shift_d;                      // log2(d / 8)
};

__global__ void __launch_bounds__(256) kv_preflight_kernel(const KvArgs a) {
    gdn::grid_dep_launch();
    const int s = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (s >= a.S) return;
    const int n0 = a.node_off[s], n1 = a.node_off[s + 1], acc = a.accepted[s], n = n1 - n0;
    int err = 0;
    if (n0 < 0 || n1 < n0 || n1 > a.N || (s == 0 && n0 != 0) || (s == a.S - 1 && n1 != a.N) || n > a.max_tokens) {
        err = GDN_DEV_BAD_NODE_OFF;
    } else if (acc < -1 || acc >= n) {
        err = GDN_DEV_BAD_ACCEPTED;
    } else if (acc >= 0) {
        const int p_lo = lane < n ? a.parents[n0 + lane] : -1;
        const int p_hi = lane + 32 < n ? a.parents[n0 + lane + 32] : -1;
        for (int cur = acc; cur >= 0 && !err;) {
            const int p = __shfl_sync(0xffffffffu, cur < 32 ? p_lo : p_hi, cur & 31);
            if (p < -1 || p >= cur) err = GDN_DEV_BAD_PARENT;
            cur = p;
        }
    }
    gdn::grid_dep_wait();  // ctx_len, the page table, status
    const int ctx = a.ctx_len[s];
    if (!err) {
        if (ctx < 0 || int64_t(ctx) + n > (int64_t(a.pl.width) << a.pl.shift)) {
            err = GDN_DEV_BAD_LEN;
        } else if (acc >= 0) {
            // the pages of positions ctx .. ctx + acc: at most 64 / 8 + 1
            bool bad = false;
            const int g = (ctx >> a.pl.shift) + lane;
            if (g <= (ctx + acc) >> a.pl.shift) {
                const int page = a.pl.table[int64_t(s) * a.pl.width + g];
                bad = page < 0 || page >= a.pl.n_pages;
            }
            if (__any_sync(0xffffffffu, bad)) err = GDN_DEV_BAD_PAGE;
        }
    }
    if (err && lane == 0) gdn::record_status(a.status, err);
}

__global__ void __launch_bounds__(256) kv_move_kernel(const KvArgs a) {
    __shared__ int64_t from[gdn::kMaxSeqNodes], to[gdn::kMaxSeqNodes];
    __shared__ int m_s;
    gdn::grid_dep_launch();
    const int s = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    gdn::grid_dep_wait();
    if (*reinterpret_cast<volatile int32_t *>(a.status) != 0) return;
    const int acc = a.accepted[s], n0 = a.node_off[s], ctx = a.ctx_len[s];
    if (tid < 32) {
        // the path, leaf first by shuffles, as a mask of nodes: rank in the mask = place
        int m = 0;
        if (acc >= 0) {
            const int p_lo = lane <= acc ? a.parents[n0 + lane] : -1;
            const int p_hi = lane + 32 <= acc ? a.parents[n0 + lane + 32] : -1;
            unsigned long long path = 0;
            for (int cur = acc; cur >= 0;) {
                path |= 1ull << cur;
                cur = __shfl_sync(0xffffffffu, cur < 32 ? p_lo : p_hi, cur & 31);
            }
            m = __popcll(path);
            for (int x = lane; x <= acc; x += 32) {
                if (!((path >> x) & 1)) continue;
                const int j = __popcll(path & ((1ull << x) - 1));
                from[j] = j == x ? -1 : gdn::position_offset(a.pl, s, ctx + x);  // -1: in place already
                to[j] = gdn::position_offset(a.pl, s, ctx + j);
            }
        }
        if (lane == 0) {
            m_s = m;
            if (layer == 0 && blockIdx.z == 0) a.new_len[s] = ctx + m;
        }
    }
    __syncthreads();
    const int m = m_s;
    const int c = blockIdx.z * blockDim.x + tid;
    if (m == 0 || c >= 2 * a.cols) return;
    const bool is_v = c >= a.cols;
    const int col = is_v ? c - a.cols : c;
    // 16-bit elements; a column is 8 of them
    uint16_t *pool = static_cast<uint16_t *>(is_v ? a.v_pool : a.k_pool) + layer * a.layer_stride +
                     int64_t(col >> a.shift_d) * a.pl.head_stride + int64_t(col & ((1 << a.shift_d) - 1)) * 8;
    for (int j0 = 0; j0 < m; j0 += 8) {
        uint4 r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < m && from[j0 + j] >= 0) r[j] = *reinterpret_cast<const uint4 *>(pool + from[j0 + j]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < m && from[j0 + j] >= 0) *reinterpret_cast<uint4 *>(pool + to[j0 + j]) = r[j];
    }
}

// Whether no two layers share a row: a thread moves its layer's rows in place, so a row of another layer must not
// be among them.  What has a smaller stride than the layers' lies within it, what has a larger one beyond all layers.
bool layers_apart(const gdn_attn_dims *d, int n_layers, int64_t layer_stride) {
    const int64_t stride[3] = {d->page_stride, d->token_stride, d->head_stride};
    const int64_t count[3] = {d->n_pages, d->page_size, d->h_kv};
    double span = d->d_head;  // (an int64 may not hold what dims of no real cache give)
    for (int k = 0; k < 3; ++k)
        if (count[k] > 1 && stride[k] < layer_stride) span += double(count[k] - 1) * double(stride[k]);
    if (double(layer_stride) < span) return false;
    span += double(n_layers - 1) * double(layer_stride);
    for (int k = 0; k < 3; ++k)
        if (count[k] > 1 && stride[k] >= layer_stride && double(stride[k]) < span) return false;
    return true;
}

}  // namespace

extern "C" int gdn_kv_commit(const gdn_attn_dims *dims, int n_layers, int64_t layer_stride, const int32_t *accepted,
                             const int32_t *parents, const int32_t *node_off, const int32_t *ctx_len,
                             const int32_t *page_table, void *k_pool, void *v_pool, int32_t *new_len, int32_t *status,
                             void *stream) {
    int rc = gdn::check_attn_dims(dims);
    if (rc) return rc;
    if (!status) return GDN_ERR_NULL;
    if (dims->max_seq_tokens > gdn::kMaxSeqNodes) return GDN_ERR_DIMS;
    if (n_layers < 0 || n_layers > 65535) return GDN_ERR_ARG;
    const int64_t S = dims->n_seqs, N = dims->n_tokens;
    if (S == 0 || n_layers == 0) return GDN_OK;
    if (!accepted || !node_off || !ctx_len || !page_table || !k_pool || !v_pool || !new_len || (N > 0 && !parents))
        return GDN_ERR_NULL;
    if (layer_stride < 0 || layer_stride % 8 != 0 || layer_stride > (int64_t(1) << 38)) return GDN_ERR_STRIDE;
    if (n_layers > 1 && !layers_apart(dims, n_layers, layer_stride)) return GDN_ERR_STRIDE;
    if (!gdn::aligned16(k_pool) || !gdn::aligned16(v_pool)) return GDN_ERR_ALIGN;
    const size_t pool = size_t(layer_stride) * 2 * size_t(n_layers - 1) + gdn::pool_bytes(dims);
    const gdn::Span ins[] = {{accepted, size_t(S * 4)},
                             {parents, size_t(N * 4)},
                             {node_off, size_t((S + 1) * 4)},
                             {ctx_len, size_t(S * 4)},
                             {page_table, size_t(S * int64_t(dims->table_width) * 4)},
                             {status, 4}};
    const gdn::Span ko[] = {{k_pool, pool}, {new_len, size_t(S * 4)}}, vo[] = {{v_pool, pool}, {new_len, size_t(S * 4)}};
    if ((rc = gdn::check_alias(ko, 2, ins, 6)) || (rc = gdn::check_alias(vo, 2, ins, 6))) return rc;

    const int cols = dims->h_kv * dims->d_head / 8;
    KvArgs a{accepted, parents, node_off, ctx_len, gdn::paged_layout(dims, page_table), k_pool, v_pool, layer_stride,
             new_len, status, int(S), int(N), dims->max_seq_tokens, dims->h_kv, cols,
             dims->d_head == 64 ? 3 : dims->d_head == 128 ? 4 : 5};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (gdn::launch_pdl(kv_preflight_kernel, dim3(unsigned((S + 7) / 8)), dim3(256), 0, st, a) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    const int threads = 2 * cols < 256 ? ((2 * cols + 31) & ~31) : 256;
    const dim3 grid(unsigned(S), unsigned(n_layers), unsigned((2 * cols + threads - 1) / threads));
    return gdn::launch_pdl(kv_move_kernel, grid, dim3(unsigned(threads)), 0, st, a) == cudaSuccess ? GDN_OK
                                                                                                     : GDN_ERR_LAUNCH;
}
