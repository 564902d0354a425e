// gdn_kv4.h - the paged cache held in 4 bits: dims checks, the places of rows in
// it, and its formats' conversions.  Not part of the public ABI.
//
// 16 elements share an e4m3 scale; a block (page, head) is page_size rows of d / 2
// bytes of e2m1 codes, then page_size rows of d / 16 scales, so that a page's keys
// of one head are one contiguous run of bytes, and so are a tile's codes.
#pragma once

#include <cmath>

#include "gdn_attn.h"

namespace gdn {

inline int64_t kv4_block(const gdn_attn_dims *d) { return int64_t(d->page_size) * d->d_head / 16 * 9; }

inline int check_kv4_dims(const gdn_attn_dims *d) {
    const int rc = check_attn_shape(d);
    if (rc) return rc;
    const int64_t s[2] = {d->page_stride, d->head_stride};
    for (int64_t x : s)
        if (x < kv4_block(d) || x % 16 != 0 || x > (int64_t(1) << 38)) return GDN_ERR_STRIDE;
    return GDN_OK;
}

inline size_t kv4_pool_bytes(const gdn_attn_dims *d) {
    return static_cast<size_t>(int64_t(d->n_pages - 1) * d->page_stride + int64_t(d->h_kv - 1) * d->head_stride +
                               kv4_block(d));
}

inline bool good_unit(float u) {
    int e;
    return std::isfinite(u) && u > 0.f && std::frexp(u, &e) == 0.5f && e - 1 >= -24 && e - 1 <= 24;
}

// Where a pool holds a position's row: codes and scales, in bytes from the pool's start.
struct Kv4Layout {
    const int32_t *__restrict__ table;
    int width, n_pages, shift;  // page_size = 1 << shift
    int64_t page_stride, head_stride;
    int code_row, scale_row;  // bytes: d / 2, d / 16
};

inline Kv4Layout kv4_layout(const gdn_attn_dims *d, const int32_t *table) {
    int shift = 0;
    while ((1 << shift) < d->page_size) ++shift;
    return {table, d->table_width, d->n_pages, shift, d->page_stride, d->head_stride, d->d_head / 2, d->d_head / 16};
}

// The page of position x of sequence s; -1 for one outside the pool.
__device__ __forceinline__ int kv4_page(const Kv4Layout &p, int s, int x) {
    const int page = p.table[int64_t(s) * p.width + (x >> p.shift)];
    return page < 0 || page >= p.n_pages ? -1 : page;
}
__device__ __forceinline__ int64_t kv4_codes(const Kv4Layout &p, int x) {
    return int64_t(x & ((1 << p.shift) - 1)) * p.code_row;
}
__device__ __forceinline__ int64_t kv4_scales(const Kv4Layout &p, int x) {
    return (int64_t(p.code_row) << p.shift) + int64_t(x & ((1 << p.shift) - 1)) * p.scale_row;
}

// Two e2m1 codes (a byte, the first in its low half) as fp16, exactly.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(byte));
    return r;
}
// Two floats as e2m1 codes, to nearest (ties to even), 6 at most; x in the low half.
__device__ __forceinline__ uint32_t to_e2m1x2(float x, float y) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(x), "f"(y));
    return r;
}
// Two e4m3 (the low 16 bits) as fp16, exactly; 0x7f is NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
// A float >= 0 as e4m3, to nearest (ties to even), 448 at most.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}
constexpr uint32_t kNanScale = 0x7f;

}  // namespace gdn
