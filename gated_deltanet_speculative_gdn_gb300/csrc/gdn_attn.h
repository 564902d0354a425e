// gdn_attn.h - what the attention layers' entry points share: dims checks, byte
// spans of the paged pools, and the places of positions in them.  Not part of
// the public ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {

inline int check_attn_dims(const gdn_attn_dims *d) {
    if (!d) return GDN_ERR_NULL;
    if (d->n_seqs < 0 || d->n_seqs > 65535 || d->n_tokens < 0 || d->max_seq_tokens < 1) return GDN_ERR_DIMS;
    if (d->h_kv < 1 || d->h_kv > 65535 || d->h_q < d->h_kv || d->h_q % d->h_kv != 0 || d->h_q / d->h_kv > 128 || d->h_q > 65535)
        return GDN_ERR_DIMS;
    if (d->d_head != 64 && d->d_head != 128 && d->d_head != 256) return GDN_ERR_DIMS;
    if (d->dtype != GDN_BF16 && d->dtype != GDN_FP16) return GDN_ERR_DIMS;
    if (d->n_pages < 1 || d->table_width < 1) return GDN_ERR_DIMS;
    if (d->page_size < 8 || d->page_size > 1024 || (d->page_size & (d->page_size - 1))) return GDN_ERR_DIMS;
    // positions are int32
    if (static_cast<int64_t>(d->table_width) * d->page_size > INT32_MAX - 65536) return GDN_ERR_DIMS;
    if (static_cast<int64_t>(d->n_tokens) * d->h_q * d->d_head > (int64_t(1) << 40)) return GDN_ERR_DIMS;
    const int64_t s[3] = {d->page_stride, d->token_stride, d->head_stride};
    for (int64_t x : s)
        if (x < d->d_head || x % 8 != 0 || x > (int64_t(1) << 38)) return GDN_ERR_STRIDE;
    return GDN_OK;
}

inline size_t rows_bytes16(int64_t rows, int64_t stride, int64_t width) {
    return rows <= 0 ? 0 : static_cast<size_t>(((rows - 1) * stride + width) * 2);
}

// Rows of `width` 16-bit elements, `stride` apart.
struct Rows16 {
    const void *p;
    int64_t stride, width;
};
inline Span span(const Rows16 &r, int64_t rows) { return {r.p, rows_bytes16(rows, r.stride, r.width)}; }

// Whether two sets of as many rows share a byte.  With one stride, so columns of one buffer as a rule, their places
// within a stride say so; with two the spans from the first row to the last must be apart.
inline bool rows_overlap(const Rows16 &a, const Rows16 &b, int64_t rows) {
    if (!overlaps(span(a, rows), span(b, rows))) return false;
    if (a.stride != b.stride) return true;
    const int64_t s = 2 * a.stride;
    int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % s;
    if (at < 0) at += s;  // b's place within a's stride
    return at < 2 * a.width || at + 2 * b.width > s;
}

inline size_t pool_bytes(const gdn_attn_dims *d) {
    return static_cast<size_t>((int64_t(d->n_pages - 1) * d->page_stride + int64_t(d->page_size - 1) * d->token_stride +
                                int64_t(d->h_kv - 1) * d->head_stride + d->d_head) * 2);
}

// Where the paged pools hold a position.
struct PagedLayout {
    const int32_t *__restrict__ table;
    int width, n_pages, shift;  // page_size = 1 << shift
    int64_t page_stride, token_stride, head_stride;
};

inline PagedLayout paged_layout(const gdn_attn_dims *d, const int32_t *table) {
    int shift = 0;
    while ((1 << shift) < d->page_size) ++shift;
    return {table, d->table_width, d->n_pages, shift, d->page_stride, d->token_stride, d->head_stride};
}

// Element offset of (position x of sequence s, head 0); -1 for a page index
// outside the pool.  x < table_width * page_size.
__device__ __forceinline__ int64_t position_offset(const PagedLayout &p, int s, int x) {
    const int page = p.table[int64_t(s) * p.width + (x >> p.shift)];
    if (page < 0 || page >= p.n_pages) return -1;
    return int64_t(page) * p.page_stride + int64_t(x & ((1 << p.shift) - 1)) * p.token_stride;
}

// Two 16-bit values in a word as floats, and back (round to nearest even).
template <typename T> struct Half2;
template <> struct Half2<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
        return r;
    }
};
template <> struct Half2<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) { return unpack_f16x2(w); }
    static __device__ __forceinline__ uint32_t pack(float x, float y) { return pack_f16x2(x, y); }
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Half2<T>::unpack(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(Half2<T>::pack(x[0], x[1]), Half2<T>::pack(x[2], x[3]), Half2<T>::pack(x[4], x[5]),
                      Half2<T>::pack(x[6], x[7]));
}

// Warp-collective: the sequence of token n, i.e. the last s in [0, S) with
// node_off[s] <= n (0 when there is none); 32 boundaries are probed at a time.
__device__ __forceinline__ int find_sequence(const int32_t *node_off, int S, int n) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = S;  // the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < hi && node_off[at] <= n);
        lo += __popc(m) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Threads t of n check all of node_off (each its share); GDN_DEV_BAD_NODE_OFF or 0.
__device__ __forceinline__ int check_node_off(const int32_t *node_off, int S, int N, int max_tokens, int t, int n) {
    bool bad = t == 0 && (node_off[0] != 0 || node_off[S] != N);
    for (int s = t; s < S; s += n) {
        const int a = node_off[s], b = node_off[s + 1];
        bad |= a < 0 || b < a || b > N || b - a > max_tokens;
    }
    return bad ? GDN_DEV_BAD_NODE_OFF : 0;
}

}  // namespace gdn
