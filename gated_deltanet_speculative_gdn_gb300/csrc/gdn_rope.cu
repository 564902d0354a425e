// gdn_rope.cu - q/k RMS norm, rotary positions with several axes, and the append
// of the new tokens' keys and values to the paged cache: what a full-attention
// layer of a hybrid model does before its attention.
//
// Mathematics.  A pair (y_a, y_b) is turned by phi = pos * f.  Far positions need
// phi mod 2 pi to more than fp32: with f / (2 pi) mod 1 as a 64-bit fraction F,
// the product pos * F wraps modulo 2^64, which is the reduction modulo one turn
// itself, exact but for F's own rounding (2^-64).  The top 32 bits, as a signed
// fraction, go to sincospif.  F comes from f's mantissa by one integer product:
// in fp64 arithmetic (1/64 of the fp32 rate here) it took most of the kernel's time.
//
// Mapping.  A warp takes one token and a share of its rows (q heads, k heads, v
// heads); a lane holds 8 elements (128-bit loads and stores), so a row of d takes
// d / 8 lanes and 256 / d rows go at a time.  The pair partner of a lane's 8
// elements is a whole lane away (rot_dim is a multiple of 16), fetched by
// shuffles.  The sines and cosines are formed once per token and warp and stay in
// registers over its rows.  Each row is read and written once: 10,004 tokens of 16 + 2 + 2
// rows of 256 take 45 us (4.5 TB/s of the copy's 6.8), held back by latency: a warp's look-ups,
// angles and batches of rows follow one another, and no batch is requested before the last one
// is stored.  (Issue slots are 56 % busy, and loads are what is waited for most.)  More warps
// spill (46 us), eight rows in flight a warp leave fewer warps (52 us).
#include "gdn_attn.h"

namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 4;  // rows of a warp in flight

// f mod 2 pi, f finite and >= 0, as a 64-bit fraction of a turn.  f = m 2^(e - 52) with a
// 53-bit m; f / (2 pi) 2^64 = m R 2^(e - 52) with R = 2^64 / (2 pi).
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
    constexpr unsigned long long R = 0x28be60db9391054aull;
    const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(f));
    const int be = int((b >> 52) & 0x7ff);
    const unsigned long long m = (b & 0xfffffffffffffull) | (be ? 1ull << 52 : 0);
    const int shift = 52 - ((be ? be : 1) - 1023);  // to the right
    const unsigned long long hi = __umul64hi(m, R), lo = m * R;
    unsigned long long r;
    if (shift >= 128) r = 0;
    else if (shift >= 64) r = hi >> (shift - 64);
    else if (shift > 0) r = (lo >> shift) | (hi << (64 - shift));
    else r = shift > -64 ? lo << -shift : 0;
    return b >> 63 ? 0ull - r : r;
}

struct RopeArgs {
    const void *__restrict__ q, *__restrict__ k, *__restrict__ v;
    int64_t q_stride, k_stride, v_stride, qo_stride;
    const float *__restrict__ qw, *__restrict__ kw;
    float eps;
    const int32_t *__restrict__ pos;
    const double *__restrict__ inv_freq;
    const int32_t *__restrict__ axis;
    int n_axes, rot, interleaved;
    const int32_t *__restrict__ node_off, *__restrict__ ctx_len;
    gdn::PagedLayout pl;
    void *qo;
    void *k_pool, *v_pool;
    int32_t *status;
    int S, N, max_tokens, Hq, Hkv, shares;  // shares: warps of a token
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 6) rope_append_kernel(const RopeArgs a) {
    constexpr int LH = D / 8, RW = 32 / LH;  // lanes of a row, rows of a warp
    const unsigned full = 0xffffffffu;
    gdn::grid_dep_launch();
    const int lane = threadIdx.x & 31, sub = lane / LH, l = lane % LH;
    const int64_t wid = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (blockIdx.x == 0) {
        const int err = gdn::check_node_off(a.node_off, a.S, a.N, a.max_tokens, threadIdx.x, kWarps * 32);
        gdn::grid_dep_wait();
        if (err) gdn::record_status(a.status, err);
    } else {
        gdn::grid_dep_wait();
    }
    const int n = int(wid / a.shares), share = int(wid % a.shares);
    if (n >= a.N) return;
    const int col = 8 * l;
    const int s = gdn::find_sequence(a.node_off, a.S, n);
    const int n0 = a.node_off[s], ctx = a.ctx_len[s];
    const int i = n - n0;
    int64_t place = -1;  // element offset of the token in the pools
    {
        int err = 0;
        const int64_t x = int64_t(ctx) + i;
        if (i < 0 || i >= a.max_tokens || n >= a.node_off[s + 1]) {
            err = GDN_DEV_BAD_NODE_OFF;
        } else if (ctx < 0 || x >= (int64_t(a.pl.width) << a.pl.shift)) {
            err = GDN_DEV_BAD_LEN;
        } else {
            place = gdn::position_offset(a.pl, s, int(x));
            if (place < 0) err = GDN_DEV_BAD_PAGE;
        }
        if (err && lane == 0) gdn::record_status(a.status, err);
    }

    // Each frequency once a warp: lane p % 32 forms pair p's cosine and sine, then every lane fetches those
    // of its eight elements (element e is column 8 l + e).
    const int half = a.rot / 2;
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
    }
    const bool turned = col < a.rot;
    const bool upper = !a.interleaved && col >= half;  // the lane holds second elements of pairs
    const int p0 = a.interleaved ? col / 2 : (upper ? col - half : col);
    bool bad = false;
    for (int k = 0; 32 * k < half; ++k) {
        const int p = 32 * k + lane;
        float c = 1.f, sv = 0.f;
        if (p < half) {
            int ax = a.axis ? a.axis[p] : 0;
            if (ax < 0 || ax >= a.n_axes) {
                bad = true;
                ax = 0;
            }
            const unsigned long long turns =
                static_cast<unsigned long long>(static_cast<long long>(a.pos[int64_t(n) * a.n_axes + ax])) *
                turn_fraction(a.inv_freq[p]);
            // a signed 32-bit fraction of a turn, in units of half turns
            sincospif(float(int(turns >> 32)) * (1.0f / 2147483648.0f), &sv, &c);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int q = p0 + (a.interleaved ? e / 2 : e);
            const float fc = __shfl_sync(full, c, q & 31), fs = __shfl_sync(full, sv, q & 31);
            if (turned && q >> 5 == k) {
                cs[e] = fc;
                sn[e] = fs;
            }
        }
    }
    if (bad) gdn::record_status(a.status, GDN_DEV_BAD_AXIS);
    // the first of a pair takes the other's share away
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (a.interleaved ? (e & 1) == 0 : !upper) sn[e] = -sn[e];
    const int hop = a.rot / 16;  // lanes between the halves of a pair
    const int partner = turned && !a.interleaved ? (upper ? lane - hop : lane + hop) : lane;

    // The rows of one kind, RW heads at a time, this warp's slots of them: kBatch rows are in flight.
    // first: the kind's first slot in the token's numbering (q, k, v).
    auto rows_of = [&](const T *src, int heads, int first, const float *w, bool turn, T *dst, int64_t dst_head) {
        const int slots = (heads + RW - 1) / RW;
        int j = share - first % a.shares;
        if (j < 0) j += a.shares;
        if (j >= slots) return;
        float wv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) wv[e] = w ? w[col + e] : 1.f;
        for (; j < slots; j += kBatch * a.shares) {
            uint4 raw[kBatch];
#pragma unroll
            for (int z = 0; z < kBatch; ++z) {
                const int r = (j + z * a.shares) * RW + sub;
                raw[z] = r < heads ? *reinterpret_cast<const uint4 *>(src + r * D + col) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int z = 0; z < kBatch; ++z) {
                const int r = (j + z * a.shares) * RW + sub;
                uint4 out = raw[z];
                if (turn) {
                    float y[8], x[8];
                    gdn::unpack8<T>(raw[z], y);
                    if (w) {
                        float ss = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
                        for (int o = LH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(full, ss, o);
                        const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * wv[e];
                    }
                    if (a.interleaved) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = fmaf(y[e ^ 1], sn[e], y[e] * cs[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = fmaf(__shfl_sync(full, y[e], partner), sn[e], y[e] * cs[e]);
                    }
                    // untouched values are copied, not converted: a NaN keeps its bits
                    if (turned || w) out = gdn::pack8<T>(x);
                }
                if (r < heads && dst) *reinterpret_cast<uint4 *>(dst + r * dst_head + col) = out;
            }
        }
    };
    const int sq = (a.Hq + RW - 1) / RW, sk = (a.Hkv + RW - 1) / RW;
    rows_of(static_cast<const T *>(a.q) + n * a.q_stride, a.Hq, 0, a.qw, a.rot > 0 || a.qw,
            static_cast<T *>(a.qo) + n * a.qo_stride, D);
    rows_of(static_cast<const T *>(a.k) + n * a.k_stride, a.Hkv, sq, a.kw, a.rot > 0 || a.kw,
            place >= 0 ? static_cast<T *>(a.k_pool) + place : nullptr, a.pl.head_stride);
    rows_of(static_cast<const T *>(a.v) + n * a.v_stride, a.Hkv, sq + sk, nullptr, false,
            place >= 0 ? static_cast<T *>(a.v_pool) + place : nullptr, a.pl.head_stride);
}

template <typename T>
cudaError_t launch(int d, dim3 grid, cudaStream_t st, const RopeArgs &a) {
    const dim3 block(kWarps * 32);
    switch (d) {
        case 64: return gdn::launch_pdl(rope_append_kernel<T, 64>, grid, block, 0, st, a);
        case 128: return gdn::launch_pdl(rope_append_kernel<T, 128>, grid, block, 0, st, a);
        default: return gdn::launch_pdl(rope_append_kernel<T, 256>, grid, block, 0, st, a);
    }
}

}  // namespace

extern "C" int gdn_rope_append(const gdn_attn_dims *dims, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                               const void *v, int64_t v_stride, const float *q_norm_w, const float *k_norm_w, float eps,
                               const int32_t *pos, int n_axes, const double *inv_freq, const int32_t *axis, int rot_dim,
                               int interleaved, const int32_t *node_off, const int32_t *ctx_len, const int32_t *page_table,
                               void *q_out, int64_t q_out_stride, void *k_pool, void *v_pool, int32_t *status,
                               void *stream) {
    int rc = gdn::check_attn_dims(dims);
    if (rc) return rc;
    if (!status) return GDN_ERR_NULL;
    if (rot_dim < 0 || rot_dim > dims->d_head || rot_dim % 16 != 0 || n_axes < 1 || n_axes > 4 ||
        (interleaved != 0 && interleaved != 1) || !(eps >= 0.0f) || !(eps < 3.0e38f))
        return GDN_ERR_ARG;
    const int64_t S = dims->n_seqs, N = dims->n_tokens, Hq = dims->h_q, Hkv = dims->h_kv, D = dims->d_head;
    if (S == 0 || N == 0) return GDN_OK;
    if (!q || !k || !v || !node_off || !ctx_len || !page_table || !q_out || !k_pool || !v_pool) return GDN_ERR_NULL;
    if (rot_dim > 0 && (!pos || !inv_freq)) return GDN_ERR_NULL;
    if (q_stride < Hq * D || k_stride < Hkv * D || v_stride < Hkv * D || q_out_stride < Hq * D || q_stride % 8 ||
        k_stride % 8 || v_stride % 8 || q_out_stride % 8)
        return GDN_ERR_STRIDE;
    if (!gdn::aligned16(q) || !gdn::aligned16(k) || !gdn::aligned16(v) || !gdn::aligned16(q_out) ||
        !gdn::aligned16(k_pool) || !gdn::aligned16(v_pool) || !gdn::aligned16(q_norm_w) || !gdn::aligned16(k_norm_w) ||
        (reinterpret_cast<uintptr_t>(inv_freq) & 7u))
        return GDN_ERR_ALIGN;
    const size_t pool = gdn::pool_bytes(dims);
    const gdn::Rows16 qr{q, q_stride, Hq * D}, kr{k, k_stride, Hkv * D}, vr{v, v_stride, Hkv * D},
        qor{q_out, q_out_stride, Hq * D};
    const gdn::Span qos = gdn::span(qor, N);
    const gdn::Span ins[] = {{q_norm_w, size_t(D * 4)},
                             {k_norm_w, size_t(D * 4)},
                             {pos, size_t(N * n_axes * 4)},
                             {inv_freq, size_t(rot_dim * 4)},
                             {axis, size_t(rot_dim * 2)},
                             {node_off, size_t((S + 1) * 4)},
                             {ctx_len, size_t(S * 4)},
                             {page_table, size_t(S * int64_t(dims->table_width) * 4)},
                             {status, 4}};
    // the pools may interleave, so they are not checked against each other
    const gdn::Span ko[] = {{k_pool, pool}, qos}, vo[] = {{v_pool, pool}, qos};
    if ((rc = gdn::check_alias(ko, 2, ins, 9)) || (rc = gdn::check_alias(vo, 2, ins, 9))) return rc;
    for (const gdn::Rows16 &r : {qr, kr, vr})
        if (gdn::overlaps(gdn::span(r, N), ko[0]) || gdn::overlaps(gdn::span(r, N), vo[0])) return GDN_ERR_ALIAS;
    // q, k, v and q_out may be columns of one buffer, so their rows are looked at, not the spans from first to last
    if (gdn::rows_overlap(qor, kr, N) || gdn::rows_overlap(qor, vr, N)) return GDN_ERR_ALIAS;
    if (gdn::rows_overlap(qor, qr, N) && !(q == q_out && q_stride == q_out_stride)) return GDN_ERR_ALIAS;

    // a token's rows are shared by as many warps as it takes to fill the GPU
    // when there are few tokens; a warp with all rows of a token forms the
    // angles once for all of them
    const int64_t rw = 256 / D, slots = (Hq + rw - 1) / rw + 2 * ((Hkv + rw - 1) / rw);
    const int64_t want = 152 * 24;
    const int64_t shares = N >= want ? 1 : (want / N < slots ? want / N : slots);
    RopeArgs a{q, k, v, q_stride, k_stride, v_stride, q_out_stride, q_norm_w, k_norm_w, eps, pos, inv_freq, axis,
               n_axes, rot_dim, interleaved, node_off, ctx_len, gdn::paged_layout(dims, page_table), q_out, k_pool, v_pool,
               status, int(S), int(N), dims->max_seq_tokens, int(Hq), int(Hkv), int(shares)};
    const dim3 grid(unsigned((N * shares + kWarps - 1) / kWarps));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dims->dtype == GDN_BF16 ? launch<__nv_bfloat16>(int(D), grid, st, a)
                                                  : launch<__half>(int(D), grid, st, a);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
