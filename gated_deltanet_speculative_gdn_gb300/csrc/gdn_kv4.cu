// gdn_kv4.cu - rows into the 4-bit cache and out of it.
//
// Mathematics.  s = e4m3(max |x| / 6 unit), code = e2m1(x / (s unit)), of the exact
// quotients.  x has 11 significant bits at most, so many quotients stand exactly on
// the border between two codes, and none other comes near one:
//   max |x| / 6 unit is formed by fp32 division.  A border B of e4m3 has 5 bits; 6 B
//     has 7, so a quotient that is no border is 2^-11 of it away at least, and fp32's
//     rounding (2^-24) neither reaches nor passes it.
//   x / (s unit) is x r, r the fp32 reciprocal, rounded to a multiple of 2^-14 (by
//     adding 768 and taking it away): off by 2^-15 + 2^-20.  A border B = b / 4 is such
//     a multiple, so a quotient on it arrives on it.  One off it is off by
//     |x - B s unit| / (s unit), whose numerator is a multiple of x's last bit, 2^-11
//     of x at least (so the quotient off by B 2^-11 >= 2^-13), or of 1/4 of s's last
//     bit (1/60): it stays on its side.
//
// Mapping.  A warp takes one token and 32 of its 16-element groups (both of keys and
// values, all heads), a thread one group: 32 bytes in, 8 and 1 out, neighbours side by
// side.  Bound by latency: append and read of 64 tokens (2 heads of 256) take 5.0 us in a
// graph, two launches; of 10,004 tokens 17.5 us, 52 MB at 3.0 TB/s, where a thread's one load, its
// conversions (two divisions) and its stores are not overlapped with another's but by occupancy.
#include <type_traits>

#include "gdn_kv4.h"

namespace {

constexpr int kWarps = 4;

struct Kv4Args {
    const void *k_in, *v_in;
    void *k_out, *v_out;
    int64_t k_stride, v_stride;  // elements between tokens' rows
    float k_unit, v_unit;
    const int32_t *__restrict__ node_off, *__restrict__ at;  // at: the position of a sequence's first token
    gdn::Kv4Layout pl;
    void *k_pool, *v_pool;
    int64_t layer_stride;  // bytes
    int32_t *status;
    int S, N, max_tokens, Hkv, parts;  // parts: warps of a token
};

// The token of this warp and the 16-element group of this thread.
struct Place {
    bool ok;       // there is a group, and its place in the cache is in order
    int n, g;      // token; group in its row
    bool is_v;
    int64_t codes, scale;  // bytes from the pool's start
};

__device__ __forceinline__ Place find_place(const Kv4Args &a, int64_t wid) {
    Place p{false, 0, 0, false, 0, 0};
    const int lane = threadIdx.x & 31;
    if (wid >= int64_t(a.N) * a.parts) return p;  // whole warps
    p.n = int(wid / a.parts);
    const int s = gdn::find_sequence(a.node_off, a.S, p.n);
    const int n0 = a.node_off[s], i = p.n - n0, per_head = a.pl.scale_row;
    const int64_t x = int64_t(a.at[s]) + i;
    int err = 0, page = -1;
    if (i < 0 || i >= a.max_tokens || p.n >= a.node_off[s + 1]) err = GDN_DEV_BAD_NODE_OFF;
    else if (x < i || x >= (int64_t(a.pl.width) << a.pl.shift)) err = GDN_DEV_BAD_LEN;
    else if ((page = gdn::kv4_page(a.pl, s, int(x))) < 0) err = GDN_DEV_BAD_PAGE;
    if (err) {
        if (lane == 0) gdn::record_status(a.status, err);
        return p;
    }
    const int groups = a.Hkv * per_head;
    int g = int(wid % a.parts) * 32 + lane;
    if (g >= 2 * groups) return p;
    p.ok = true;
    p.is_v = g >= groups;
    p.g = p.is_v ? g - groups : g;
    const int h = p.g / per_head, b = p.g - h * per_head;
    const int64_t block = int64_t(page) * a.pl.page_stride + int64_t(h) * a.pl.head_stride;
    p.codes = block + gdn::kv4_codes(a.pl, int(x)) + 8 * b;
    p.scale = block + gdn::kv4_scales(a.pl, int(x)) + b;
    return p;
}

__device__ __forceinline__ void first_cta_checks(const Kv4Args &a) {
    if (blockIdx.x != 0 || blockIdx.y != 0) return;
    const int err = gdn::check_node_off(a.node_off, a.S, a.N, a.max_tokens, threadIdx.x, kWarps * 32);
    if (err) gdn::record_status(a.status, err);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) kv4_append_kernel(const Kv4Args a) {
    gdn::grid_dep_launch();
    gdn::grid_dep_wait();
    first_cta_checks(a);
    const Place p = find_place(a, int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5));
    if (!p.ok) return;
    const T *row = static_cast<const T *>(p.is_v ? a.v_in : a.k_in) + p.n * (p.is_v ? a.v_stride : a.k_stride);
    const uint4 *src = reinterpret_cast<const uint4 *>(row + 16 * p.g);
    const uint4 in[2] = {src[0], src[1]};
    const float unit = p.is_v ? a.v_unit : a.k_unit;
    // the largest magnitude, as bits: infinities and NaN are above all others
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(in[i].x & 0x7fff7fffu, in[i].y & 0x7fff7fffu),
                                     __vmaxu2(in[i].z & 0x7fff7fffu, in[i].w & 0x7fff7fffu)));
    top = max(top & 0xffffu, top >> 16);
    constexpr uint32_t inf = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    uint32_t scale = gdn::kNanScale;
    uint2 codes = make_uint2(0, 0);
    if (top < inf) {
        // (unit is a power of two: the division by it is exact, or s is 0 or 448 either way)
        scale = gdn::to_e4m3(__fdiv_rn(gdn::Half2<T>::unpack(top).x / unit, 6.f));
        if (scale) {
            const float s = gdn::unpack_f16x2(gdn::e4m3x2_to_f16x2(scale)).x * unit, r = __fdiv_rn(1.f, s);
            uint32_t c[8];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float y[8];
                gdn::unpack8<T>(in[i], y);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = copysignf(__fsub_rn(__fmaf_rn(y[e], r, 768.f), 768.f), y[e]);
#pragma unroll
                for (int e = 0; e < 4; ++e) c[4 * i + e] = gdn::to_e2m1x2(y[2 * e], y[2 * e + 1]);
            }
            codes.x = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
            codes.y = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
        }
    }
    unsigned char *pool = static_cast<unsigned char *>(p.is_v ? a.v_pool : a.k_pool);
    *reinterpret_cast<uint2 *>(pool + p.codes) = codes;
    pool[p.scale] = static_cast<unsigned char>(scale);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) kv4_read_kernel(const Kv4Args a) {
    gdn::grid_dep_launch();
    gdn::grid_dep_wait();
    first_cta_checks(a);
    const Place p = find_place(a, int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5));
    if (!p.ok) return;
    const unsigned char *pool = static_cast<const unsigned char *>(p.is_v ? a.v_pool : a.k_pool) + blockIdx.y * a.layer_stride;
    const uint2 codes = *reinterpret_cast<const uint2 *>(pool + p.codes);
    const float s = gdn::unpack_f16x2(gdn::e4m3x2_to_f16x2(pool[p.scale])).x * (p.is_v ? a.v_unit : a.k_unit);
    T *row = static_cast<T *>(p.is_v ? a.v_out : a.k_out) + (int64_t(blockIdx.y) * a.N + p.n) * a.k_stride;
    uint4 *dst = reinterpret_cast<uint4 *>(row + 16 * p.g);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t c = i ? codes.y : codes.x;
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = gdn::unpack_f16x2(gdn::e2m1x2_to_f16x2((c >> (8 * e)) & 0xffu));
            y[2 * e] = f.x * s;
            y[2 * e + 1] = f.y * s;
        }
        dst[i] = gdn::pack8<T>(y);
    }
}

// What append and read check alike; GDN_OK with *empty set where there is nothing to do.
int check_common(const gdn_attn_dims *dims, float k_unit, float v_unit, const void *k, int64_t k_stride, const void *v,
                 int64_t v_stride, const int32_t *node_off, const int32_t *at, const int32_t *table, const void *k_pool,
                 const void *v_pool, const int32_t *status, bool none, bool *empty) {
    const int rc = gdn::check_kv4_dims(dims);
    if (rc) return rc;
    if (!status) return GDN_ERR_NULL;
    if (!gdn::good_unit(k_unit) || !gdn::good_unit(v_unit)) return GDN_ERR_ARG;
    *empty = none || dims->n_seqs == 0 || dims->n_tokens == 0;
    if (*empty) return GDN_OK;
    if (!k || !v || !node_off || !at || !table || !k_pool || !v_pool) return GDN_ERR_NULL;
    const int64_t row = int64_t(dims->h_kv) * dims->d_head;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8 || k_stride > (int64_t(1) << 38) ||
        v_stride > (int64_t(1) << 38))
        return GDN_ERR_STRIDE;
    if (!gdn::aligned16(k) || !gdn::aligned16(v) || !gdn::aligned16(k_pool) || !gdn::aligned16(v_pool)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

Kv4Args common_args(const gdn_attn_dims *dims, float k_unit, float v_unit, const int32_t *node_off, const int32_t *at,
                    const int32_t *table, const void *k_pool, const void *v_pool, int32_t *status) {
    Kv4Args a{};
    a.k_unit = k_unit;
    a.v_unit = v_unit;
    a.node_off = node_off;
    a.at = at;
    a.pl = gdn::kv4_layout(dims, table);
    a.k_pool = const_cast<void *>(k_pool);
    a.v_pool = const_cast<void *>(v_pool);
    a.status = status;
    a.S = dims->n_seqs;
    a.N = dims->n_tokens;
    a.max_tokens = dims->max_seq_tokens;
    a.Hkv = dims->h_kv;
    a.parts = int((2 * int64_t(dims->h_kv) * a.pl.scale_row + 31) / 32);
    return a;
}

}  // namespace

extern "C" size_t gdn_kvq_block_bytes(const gdn_attn_dims *dims) {
    return gdn::check_attn_shape(dims) == GDN_OK ? static_cast<size_t>(gdn::kv4_block(dims)) : 0;
}

extern "C" int gdn_kvq_append(const gdn_attn_dims *dims, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                              float k_unit, float v_unit, const int32_t *node_off, const int32_t *ctx_len,
                              const int32_t *page_table, void *k_pool, void *v_pool, int32_t *status, void *stream) {
    bool empty = false;
    int rc = check_common(dims, k_unit, v_unit, k, k_stride, v, v_stride, node_off, ctx_len, page_table, k_pool, v_pool,
                          status, false, &empty);
    if (rc || empty) return rc;
    const int64_t S = dims->n_seqs, N = dims->n_tokens, row = int64_t(dims->h_kv) * dims->d_head;
    const size_t pool = gdn::kv4_pool_bytes(dims);
    const gdn::Span ins[] = {{k, gdn::rows_bytes16(N, k_stride, row)},
                             {v, gdn::rows_bytes16(N, v_stride, row)},
                             {node_off, size_t((S + 1) * 4)},
                             {ctx_len, size_t(S * 4)},
                             {page_table, size_t(S * int64_t(dims->table_width) * 4)},
                             {status, 4}};
    // the pools may interleave, so they are not checked against each other
    const gdn::Span ko[] = {{k_pool, pool}}, vo[] = {{v_pool, pool}};
    if ((rc = gdn::check_alias(ko, 1, ins, 6)) || (rc = gdn::check_alias(vo, 1, ins, 6))) return rc;
    Kv4Args a = common_args(dims, k_unit, v_unit, node_off, ctx_len, page_table, k_pool, v_pool, status);
    a.k_in = k;
    a.v_in = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    const int64_t ctas = (N * a.parts + kWarps - 1) / kWarps;
    if (ctas > INT32_MAX) return GDN_ERR_DIMS;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(ctas)), block(kWarps * 32);
    const cudaError_t e = dims->dtype == GDN_BF16 ? gdn::launch_pdl(kv4_append_kernel<__nv_bfloat16>, grid, block, 0, st, a)
                                                  : gdn::launch_pdl(kv4_append_kernel<__half>, grid, block, 0, st, a);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

extern "C" int gdn_kvq_read(const gdn_attn_dims *dims, int n_layers, int64_t layer_stride, const void *k_pool,
                            const void *v_pool, float k_unit, float v_unit, const int32_t *node_off, const int32_t *start,
                            const int32_t *page_table, void *k, void *v, int64_t row_stride, int32_t *status, void *stream) {
    bool empty = false;
    int rc = check_common(dims, k_unit, v_unit, k, row_stride, v, row_stride, node_off, start, page_table, k_pool, v_pool,
                          status, n_layers == 0, &empty);
    if (rc) return rc;
    if (n_layers < 0 || n_layers > 65535) return GDN_ERR_ARG;
    if (empty) return GDN_OK;
    if (layer_stride < 0 || layer_stride % 16 != 0 || layer_stride > (int64_t(1) << 38)) return GDN_ERR_STRIDE;
    const int64_t S = dims->n_seqs, N = dims->n_tokens, row = int64_t(dims->h_kv) * dims->d_head;
    const size_t pool = size_t(layer_stride) * size_t(n_layers - 1) + gdn::kv4_pool_bytes(dims);
    const size_t rows = gdn::rows_bytes16(int64_t(n_layers) * N, row_stride, row);
    // k and v may be columns of one buffer, so their rows are looked at, not the spans from first to last
    if (gdn::rows_overlap({k, row_stride, row}, {v, row_stride, row}, int64_t(n_layers) * N)) return GDN_ERR_ALIAS;
    const gdn::Span outs[] = {{k, rows}}, outs_v[] = {{v, rows}};
    const gdn::Span ins[] = {{k_pool, pool},
                             {v_pool, pool},
                             {node_off, size_t((S + 1) * 4)},
                             {start, size_t(S * 4)},
                             {page_table, size_t(S * int64_t(dims->table_width) * 4)},
                             {status, 4}};
    if ((rc = gdn::check_alias(outs, 1, ins, 6)) || (rc = gdn::check_alias(outs_v, 1, ins, 6))) return rc;
    Kv4Args a = common_args(dims, k_unit, v_unit, node_off, start, page_table, k_pool, v_pool, status);
    a.k_out = k;
    a.v_out = v;
    a.k_stride = row_stride;
    a.layer_stride = layer_stride;
    const int64_t ctas = (N * a.parts + kWarps - 1) / kWarps;
    if (ctas > INT32_MAX) return GDN_ERR_DIMS;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(n_layers)), block(kWarps * 32);
    const cudaError_t e = dims->dtype == GDN_BF16 ? gdn::launch_pdl(kv4_read_kernel<__nv_bfloat16>, grid, block, 0, st, a)
                                                  : gdn::launch_pdl(kv4_read_kernel<__half>, grid, block, 0, st, a);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
