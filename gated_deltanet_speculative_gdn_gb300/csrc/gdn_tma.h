// gdn_tma.h - host helpers shared by the translation units that launch TMA
// kernels.  Not part of the public ABI.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "gdn.h"

namespace gdn {

// xc viewed as [N rows][C floats] with boxes of [rows][cols] floats, in the
// 128-byte swizzle when `swizzle` (the tensor cores' K-major operand layout
// for 32-float rows); GDN_OK or GDN_ERR_TMA.
int encode_xc_tiles(CUtensorMap *map, const float *xc, int64_t N, int64_t C, uint32_t rows, uint32_t cols,
                    bool swizzle);

// A paged pool of 16-bit values viewed as [page][head][d / 64][token][64], boxes of
// [chunks][rows tokens][64] of one head and page in the 128-byte swizzle; GDN_OK or GDN_ERR_TMA.
int encode_kv_pages(CUtensorMap *map, const void *pool, const gdn_attn_dims *dims, uint32_t rows, uint32_t chunks);

// Multiprocessors of the current device (0 on error).
int sm_count_current();

}  // namespace gdn
