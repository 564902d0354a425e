// gdn_attention_kvq.cu - attention over the paged cache held in 4 bits: the kernel of
// gdn_attention.cuh with keys and values that are converted on their way to the tensor
// cores (its mathematics, work and mapping are in gdn_attention.cu).
//
// Rounding.  Codes times scales have 6 significant bits and are multiples of 2^-10 up to
// 2688, so fp16 holds them exactly: both products run in fp16 whatever q's type, p rounded
// as for an fp16 cache.  fp16 q rows go in as they are, bf16 rows scaled by a power of two
// by row.  The units are factors of the scores and of the result.
//
// Mapping.  The kernel of gdn_attention.cuh with two warps that bring pages in, as they lie in
// memory, by one bulk copy each into a ring of raw tiles (the place of TMA and of cleaning), and 8
// more (4 of them working for d = 64) that convert tile after tile into the ring of fp16 tiles, in the
// 128-byte swizzle.  One conversion takes two codes and gives about 37 pairs a cycle and SM; with the
// product by the scale 72 codes a cycle and SM were measured, so a tile of keys and values at d = 256
// is ~460 cycles of conversion beside ~1,000 of products for 128 rows.  16-bit q rows go to tensor
// memory through registers.  Sequences of few rows take the second kernel.
//
// Measured: 64 trees of 16 nodes over up to 8,192 (d = 256) 97-106 us, chunks of up to 701 over up to
// 3,001 (d = 128) 309-311 (the 16-bit cache 119-122 and 262-266), 64 single tokens over up to 16,384 79
// (184-189).  Why not faster: the trees' 128 items are dealt out over 152 SMs as in the 16-bit form, so
// each SM has a start, an end and parts to write and join beside its tiles; and a tile passes conversion,
// scores, softmax and values one after the other, with few tiles under way at once (the rings hold two of
// fp16 keys and values at d = 256).  For d <= 128 the chunks are slower than over the 16-bit cache: every tile
// is converted for 128 rows only, and the rows' warps, which gave registers to the converting ones, spill 262 (fp16)
// and 278 bytes (bf16) a thread at d = 128, 182 and 196 at 64 (at 256 none and 8; the 16-bit form 104, 64 and none).
#include <type_traits>

#include "gdn_attention.cuh"

namespace {

template <typename T, int D>
__global__ void __launch_bounds__(att::Cfg<D, true>::kThreads, 1) kvq_attention_kernel(const att::Args a) {
    attention_body<T, D, true>(nullptr, nullptr, a);
}

// ---- few rows: sequences of 16 query rows of a key/value head at most, 8 for d = 256 ---------
//
// One token of a group of 8 is 8 of the 128 rows that a tensor-memory tile has, and the way
// through the roles above costs a tile as much whatever its rows: 64 single tokens over up to
// 16,384 positions take 148 us so, against 50 of memory.  Here eight warps work each by
// itself on 16 positions at a time, with the products by mma.sync on the codes as they come
// out of shared memory, converted in registers:
//     S^T[16 x rows] = K Q^T    A: keys, a lane's elements of a position one after the other
//                               (any order of d will do, as long as q has the same)
//     O^T[d x rows] += V^T P^T  A: values, whose pairs along the positions are two codes of
//                               two words put into one byte before the conversion; P^T comes
//                               out of S^T's layout by movmatrix
// so a running m and l, and O, are a warp's own until the segment ends.  m moves as in the
// other kernel.  64 single tokens take 79 us so (heads of 128: 82-85, of 64: 64), against a floor of 50 of memory
// (63 % of a copy's rate, by the times).  A warp's tile is a chain of
// shared-memory reads, conversions and products; more warps (12 of 152 registers) did not help.
// (Where it is used stands at its launch: at d = 256 a lane's q and O of 16 rows leave no registers for 32
// positions at a time.)  Four more warps copy tiles (keys and values of 64 positions) into a ring; two warps take a
// tile, four tiles are under way.  The ring has a multiple of four stages, so that each belongs to one copying warp and
// to one group: 8 of 18 KB (144 KB) at d = 256, 20 of 9 at 128, 24 of 4.5 at 64.
// At launch 168 registers a thread.  Spilled, of the working warps: 24 (fp16) and 32 bytes (bf16) at d = 256, 16 for
// 16 rows at d = 128 in bf16, none otherwise.
template <int D_, int NT_>
struct Few {
    static constexpr int D = D_, NT = NT_;                  // NT: blocks of 8 rows
    static constexpr int NS = 2;                            // strips of 16 positions that a warp takes at a time (1: 126 us for 111)
    static constexpr int kWarps = 8, kOfTile = 4 / NS, kGroups = kWarps / kOfTile, kThreads = 32 * (kWarps + 4);
    static constexpr int kCodeRow = D / 2, kScaleRow = D / 16;
    static constexpr uint32_t kRaw = att::TK * (kCodeRow + kScaleRow), kStage = 2 * kRaw;
    static constexpr int kRegs = D / 4 * NT;                // O of a lane
    static constexpr uint32_t kJoin = kOfTile * kRegs * 128;  // O of a tile's warps
    // A stage belongs to one group: its warps wait for each of its uses in turn.  (One that waited for every second use only
    // could come to a use two ahead of what has been copied, whose parity is that of the use before.)
    static constexpr int kFit = int((212992 - kJoin) / kStage), kStages = (kFit < 24 ? kFit : 24) / 4 * 4;
    static constexpr size_t kSmem = kStages * kStage + kJoin;
    static_assert(kStages >= 4 && kStages % kGroups == 0, "ring");
};

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// n consecutive 32-bit words of shared memory
template <int n>
__device__ __forceinline__ void load_words(const unsigned char *p, uint32_t (&w)[n]) {
    if constexpr (n == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (n == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < n; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[i] = v.x;
            w[i + 1] = v.y;
            w[i + 2] = v.z;
            w[i + 3] = v.w;
        }
    }
}
// n scales (1, 2 or 4 bytes)
template <int n>
__device__ __forceinline__ uint32_t load_scales(const unsigned char *p) {
    if constexpr (n == 1) return *p;
    else if constexpr (n == 2) return *reinterpret_cast<const uint16_t *>(p);
    else return *reinterpret_cast<const uint32_t *>(p);
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(Few<D, NT>::kThreads, 1) kvq_few_kernel(const att::Args a) {
    using namespace att;
    using C = Few<D, NT>;
    using Ref = Reference<__half>;
    constexpr int kThreads = C::kThreads, kWarps = C::kWarps, NS = C::NS;
    extern __shared__ __align__(128) unsigned char smem_few[];
    __shared__ uint64_t full_bar[C::kStages], empty_bar[C::kStages], never_bar;
    __shared__ int abort_s;
    __shared__ Start start_s;
    __shared__ long long wsum[kThreads / 32];
    __shared__ int tree_par[kWarps][gdn::kMaxSeqNodes];
    __shared__ float2 ml[kWarps][8 * NT];
    __shared__ uint32_t nf[2];  // by segment: which positions from `safe` on have values that are not finite
    volatile int *abort_flag = &abort_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned full = 0xffffffffu;
    unsigned char *ring = smem_few;
    float *joined = reinterpret_cast<float *>(smem_few + C::kStages * C::kStage);

    gdn::grid_dep_launch();
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            gdn::mbar_init(full_bar + i, 1);
            gdn::mbar_init(empty_bar + i, C::kOfTile);
        }
        gdn::mbar_init(&never_bar, 1);
        gdn::fence_mbar_init();
        abort_s = 0;
        start_s.count = 0;
        nf[0] = nf[1] = 0;
    }
    gdn::grid_dep_wait();
    schedule<kThreads>(a, wsum, start_s, [] { __syncthreads(); });
    __syncthreads();
    bool ok = true;
    // (the test hook: role 1 the first of the copies, the others one of the working warps)
    const int stalled = a.stall_role == 1 ? kWarps : a.stall_role;
    if (a.stall_ns && blockIdx.x == 0 && warp == stalled) {
        ok = __all_sync(full, gdn::mbar_wait_bounded(&never_bar, 0, a.stall_ns));
        if (!ok) *abort_flag = 1;
    }
    const int ps = 1 << a.pl.shift, run = raw_run(a.pl.shift);

    // 168 registers a thread at launch, 12 x 168 = 2016 of a warp's 32, shared out anew: 8 x 224 + 4 x 56 = 2016.  (Twelve working
    // warps of 152 registers gain nothing: 94 us for 87.)
    if (warp >= kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // ---- tiles, page by page, four warps in turn (one takes ~700 cycles for a tile) ------
        Walk walk(a, start_s);
        Segment g;
        asm volatile("fence.proxy.async;" ::: "memory");  // what earlier kernels wrote, for the copies
        const int runs = TK / run;
        const uint32_t codes = run * C::kCodeRow, scales = run * C::kScaleRow;
        uint32_t tiles_done = 0;
        int issued = 0, st = warp - kWarps;  // (a stage belongs to one warp)
        uint32_t phase = 0;
        bool bad_page = false;
        while (ok && walk.next(g)) {
            const int32_t *table = a.pl.table + int64_t(g.s) * a.pl.width;
            const int last = (g.limit - 1) >> a.pl.shift, n = g.tile1 - g.tile0;
            const int64_t head = int64_t(g.h) * a.pl.head_stride;
            auto page_of = [&](int k) {  // this lane's page of the segment's tile k; -1: none
                const int o = (((g.tile0 + k) * TK) >> a.pl.shift) + lane;
                return lane < runs && k < n && o <= last ? table[o] : -1;
            };
            int k = int(st % 4 + 4 - tiles_done % 4) % 4, page = page_of(k);
            for (; k < n; k += 4) {
                const int next = page_of(k + 4);  // looked up one ahead
                const int t = g.tile0 + k;
                if (page < 0 || page >= a.pl.n_pages) {
                    bad_page |= lane < runs && ((t * TK) >> a.pl.shift) + lane <= last;
                    page = -1;
                }
                ok = wait_bar(empty_bar + st, phase ^ 1, abort_flag);
                if (!ok) break;
                const bool mine = page >= 0;
                const unsigned m = __ballot_sync(full, mine);
                if (lane == 0) gdn::mbar_arrive_expect_tx(full_bar + st, __popc(m) * 2 * (codes + scales));
                __syncwarp();
                if (mine) {
                    const int at = (t * TK) & (ps - 1);
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        unsigned char *dst = ring + st * C::kStage + v * C::kRaw + lane * (codes + scales);
                        const unsigned char *block =
                            static_cast<const unsigned char *>(v ? a.v_pool : a.k_pool) + int64_t(page) * a.pl.page_stride + head;
                        if (ps == run) {
                            gdn::bulk_load(dst, block, codes + scales, full_bar + st);
                        } else {
                            gdn::bulk_load(dst, block + at * C::kCodeRow, codes, full_bar + st);
                            gdn::bulk_load(dst + codes, block + (int64_t(C::kCodeRow) << a.pl.shift) + at * C::kScaleRow, scales,
                                           full_bar + st);
                        }
                    }
                }
                page = next;
                ++issued;
                if ((st += 4) >= C::kStages) {
                    st -= C::kStages;
                    phase ^= 1;
                }
            }
            tiles_done += n;
        }
        if (bad_page) gdn::record_status(a.status, GDN_DEV_BAD_PAGE);
        // no copy is under way when the CTA leaves
        for (int z = min(issued, C::kStages / 4); z > 0; --z) {
            if ((st -= 4) < 0) {
                st += C::kStages;
                phase ^= 1;
            }
            gdn::mbar_wait_bounded(full_bar + st, phase);
        }
    } else {
        // ---- 32 positions of every fourth tile ---------------------------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        Walk walk(a, start_s);
        Segment g;
        // After a wait that ran out a warp goes on without work and without waits, so that the CTA's barriers match.
        const int gr = lane >> 2, c = lane & 3;       // the row and the pair of columns of a fragment
        const int strip = 16 * NS * (warp % C::kOfTile), group = warp / C::kOfTile;
        constexpr int KW = D / 32, VW = D / 64;       // words of codes: of a lane's part of a key, of a value
        constexpr int KS = D >= 64 ? D / 64 : 1, VS = D == 256 ? 2 : 1;  // scales of those parts
        const int piece_bytes = run * (C::kCodeRow + C::kScaleRow);
        auto codes_of = [&](int r) { return r / run * piece_bytes + r % run * C::kCodeRow; };
        auto scales_of = [&](int r) { return r / run * piece_bytes + run * C::kCodeRow + r % run * C::kScaleRow; };
        int k_at[NS][2], ks_at[NS][2], v_at[NS][4], vs_at[NS][4];
#pragma unroll
        for (int u = 0; u < NS; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = strip + 16 * u + gr + 8 * i;
                k_at[u][i] = codes_of(r) + c * (C::kCodeRow / 4);
                ks_at[u][i] = scales_of(r) + c * KS;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = strip + 16 * u + 2 * c + (i & 1) + 8 * (i >> 1);
                v_at[u][i] = int(C::kRaw) + codes_of(r) + gr * (C::kCodeRow / 8);
                vs_at[u][i] = int(C::kRaw) + scales_of(r) + gr * (D / 8) / 16;
            }
        }
        int4 *meta = a.meta + 2 * blockIdx.x;
        bool head_part = false, tail_part = false;
        uint32_t tiles_done = 0, seg = 0;  // of the CTA's tiles, before the segment
        while (walk.next(g)) {
            // ---- the segment's q, and what its rows see: rows 8 nt + gr as a fragment's, 8 nt + 2 c + e as a result's
            uint32_t q[D / 16][NT][2];
            float cr[NT][2], m[NT][2], l[NT][2], o[D / 16][NT][4];
            int upto[NT][2];
            unsigned long long line[NT][2];
            if (a.parents) {
                __syncwarp();
                for (int x = lane; x < g.q.n; x += 32) tree_par[warp][x] = a.parents[g.q.n0 + x];
                __syncwarp();
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = 8 * nt + gr;
                const bool live = row < g.rows;
                const T *src = static_cast<const T *>(a.q) + (int64_t(g.q.n0) + g.i0 + row / a.G) * a.q_stride +
                               (int64_t(g.h) * a.G + row % a.G) * D + c * (D / 4);
                uint4 v[D / 32];
#pragma unroll
                for (int i = 0; i < D / 32; ++i) v[i] = live ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
                float mine = a.c;
                if constexpr (!std::is_same<T, __half>::value) {
                    // (as in the other kernel: the row's largest element to 2^14 .. 2^15)
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                                     __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
                    top = max(top & 0xffffu, top >> 16);
                    top = max(top, __shfl_xor_sync(full, top, 1));
                    top = max(top, __shfl_xor_sync(full, top, 2));
                    const int e = int(top >> 7), s = e == 255 ? 0 : min(14 + 127 - e, 100);
                    const float f = __uint_as_float(uint32_t(127 + s) << 23);
                    mine = row_factor(a, s);
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        float y[8];
                        gdn::unpack8<T>(v[i], y);
#pragma unroll
                        for (int x = 0; x < 8; ++x) y[x] *= f;
                        v[i] = gdn::pack8<__half>(y);
                    }
                }
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    q[2 * i][nt][0] = v[i].x;
                    q[2 * i][nt][1] = v[i].y;
                    q[2 * i + 1][nt][0] = v[i].z;
                    q[2 * i + 1][nt][1] = v[i].w;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    cr[nt][e] = __shfl_sync(full, mine, 4 * (2 * c + e));
                    m[nt][e] = -INFINITY;
                    l[nt][e] = 0.f;
                    const int r = 8 * nt + 2 * c + e, i = g.i0 + r / a.G;
                    upto[nt][e] = g.q.ctx + i + 1;
                    line[nt][e] = 0;
                    if (a.parents && r < g.rows) {
                        for (int x = i; x >= 0;) {
                            line[nt][e] |= 1ull << x;
                            const int p = tree_par[warp][x];
                            if (p >= x || p < -1) {
                                gdn::record_status(a.status, GDN_DEV_BAD_PARENT);
                                break;
                            }
                            x = p;
                        }
                    }
                }
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[j][nt][e] = 0.f;
            auto sees = [&](int nt, int e, int x) {
                return a.parents ? x < g.q.ctx || (x - g.q.ctx < 64 && ((line[nt][e] >> (x - g.q.ctx)) & 1)) : x < upto[nt][e];
            };

            const int n = g.tile1 - g.tile0;
#pragma unroll 1
            for (int k = int(group + C::kGroups - tiles_done % C::kGroups) % C::kGroups; k < n; k += C::kGroups) {  // tile i of group i % kGroups
                const uint32_t i = tiles_done + k;
                const int stage = int(i % C::kStages), x0 = (g.tile0 + k) * TK + strip;
                ok = ok && wait_bar(full_bar + stage, (i / C::kStages) & 1, abort_flag);
                if (ok && x0 < g.limit) {
                    const unsigned char *src = ring + stage * C::kStage;
                    const bool masked = x0 + 16 * NS > g.safe;
                    // ---- scores: positions gr, gr + 8 of a strip by rows 2 c, 2 c + 1; two sums, of even and odd steps
                    float s[NS][2][NT][4];
#pragma unroll
                    for (int u = 0; u < NS; ++u)
#pragma unroll
                        for (int z = 0; z < 2; ++z)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) s[u][z][nt][e] = 0.f;
                    uint32_t kw[NS][2][KW], ksc[NS][2];
#pragma unroll
                    for (int u = 0; u < NS; ++u)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            load_words(src + k_at[u][r], kw[u][r]);
                            ksc[u][r] = load_scales<KS>(src + ks_at[u][r]);
                        }
#pragma unroll
                    for (int w = 0; w < KW; ++w)
#pragma unroll
                        for (int u = 0; u < NS; ++u) {
                            uint4 f[2];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const uint32_t two = gdn::e4m3x2_to_f16x2((ksc[u][r] >> (16 * (w / 4))) & 0xffffu);
                                f[r] = convert8(kw[u][r][w], __byte_perm(two, two, (w / 2) & 1 ? 0x3232 : 0x1010));
                            }
                            const uint32_t a0[4] = {f[0].x, f[1].x, f[0].y, f[1].y}, a1[4] = {f[0].z, f[1].z, f[0].w, f[1].w};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma_16816(s[u][0][nt], a0, q[2 * w][nt][0], q[2 * w][nt][1]);
                                mma_16816(s[u][1][nt], a1, q[2 * w + 1][nt][0], q[2 * w + 1][nt][1]);
                            }
                        }
                    uint32_t vw[NS][4][VW], vsc[NS][4];
#pragma unroll
                    for (int u = 0; u < NS; ++u)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            load_words(src + v_at[u][r], vw[u][r]);
                            vsc[u][r] = load_scales<VS>(src + vs_at[u][r]);
                        }
#pragma unroll
                    for (int u = 0; u < NS; ++u)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[u][0][nt][e] += s[u][1][nt][e];
                    if (masked) {
#pragma unroll
                        for (int u = 0; u < NS; ++u) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int x = x0 + 16 * u + gr + 8 * (e >> 1);
                                    if (x >= g.limit || !sees(nt, e & 1, x)) s[u][0][nt][e] = -INFINITY;
                                }
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int x = x0 + 16 * u + 2 * c + (r & 1) + 8 * (r >> 1);
                                if (x >= g.limit) {  // no row sees it
                                    vsc[u][r] = 0;
#pragma unroll
                                    for (int w = 0; w < VW; ++w) vw[u][r][w] = 0;
                                } else if (x >= g.safe) {
                                    // values that are not finite: 0 here, put back at the end for the rows that see them
#pragma unroll
                                    for (int b = 0; b < VS; ++b)
                                        if (((vsc[u][r] >> (8 * b)) & 0x7f) == gdn::kNanScale) {
                                            vsc[u][r] &= ~(0xffu << (8 * b));
                                            atomicOr(&nf[seg & 1], 1u << (x - g.safe));
                                        }
                                }
                            }
                        }
                    }
                    // ---- weights
                    auto largest = [&](int nt, int e) {
                        float x = -INFINITY;
#pragma unroll
                        for (int u = 0; u < NS; ++u) x = fmaxf(x, fmaxf(s[u][0][nt][e], s[u][0][nt][e + 2]));
                        x = fmaxf(x, __shfl_xor_sync(full, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(full, x, 8));
                        return cr[nt][e] * fmaxf(x, __shfl_xor_sync(full, x, 16));
                    };
                    bool unset = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) unset |= m[nt][0] == -INFINITY || m[nt][1] == -INFINITY;
                    if (__any_sync(full, unset)) {  // the first positions that a row sees
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float mx = largest(nt, e);
                                if (m[nt][e] == -INFINITY) m[nt][e] = mx - Ref::kLift;
                            }
                    }
                    float y[NS][NT][4], top;
                    auto exponents = [&] {
                        top = -INFINITY;
#pragma unroll
                        for (int u = 0; u < NS; ++u)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float mu = m[nt][e & 1];
                                    y[u][nt][e] = fmaf(s[u][0][nt][e], cr[nt][e & 1], mu == -INFINITY ? 0.f : -mu);
                                    top = fmaxf(top, y[u][nt][e]);
                                }
                    };
                    exponents();
                    if (__any_sync(full, top > Ref::kMoveAt)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float mx = largest(nt, e);
                                if (mx > m[nt][e] + Ref::kMoveAt) {
                                    const float f = exp2_approx(m[nt][e] - (mx - Ref::kLift));
                                    m[nt][e] = mx - Ref::kLift;
                                    l[nt][e] *= f;
#pragma unroll
                                    for (int j = 0; j < D / 16; ++j) {
                                        o[j][nt][e] *= f;
                                        o[j][nt][e + 2] *= f;
                                    }
                                }
                            }
                        exponents();
                    }
                    uint32_t pt[NS][NT][2];
#pragma unroll
                    for (int u = 0; u < NS; ++u)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float p[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) p[e] = exp2_approx(y[u][nt][e]);
                            l[nt][0] += p[0] + p[2];
                            l[nt][1] += p[1] + p[3];
                            pt[u][nt][0] = transposed(gdn::pack_f16x2(p[0], p[1]));
                            pt[u][nt][1] = transposed(gdn::pack_f16x2(p[2], p[3]));
                        }
                    // ---- values: rows of the fragment d and d + 1, pairs of positions
#pragma unroll
                    for (int u = 0; u < NS; ++u) {
                        uint32_t vs[2][VS];  // scales of positions 2 c, 2 c + 1 and 2 c + 8, 2 c + 9
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t lo = gdn::e4m3x2_to_f16x2(vsc[u][2 * z]), hi = gdn::e4m3x2_to_f16x2(vsc[u][2 * z + 1]);
                            vs[z][0] = __byte_perm(lo, hi, 0x5410);
                            if constexpr (VS == 2) vs[z][1] = __byte_perm(lo, hi, 0x7632);
                        }
#pragma unroll
                        for (int w = 0; w < VW; ++w) {
                            uint4 f[2][2];  // [low, high half of a byte][positions 2 c .., 2 c + 8 ..]
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const uint32_t w0 = vw[u][2 * z][w], w1 = vw[u][2 * z + 1][w], sc = vs[z][VS == 2 ? w / 2 : 0];
                                f[0][z] = convert8((w0 & 0x0f0f0f0fu) | ((w1 << 4) & 0xf0f0f0f0u), sc);
                                f[1][z] = convert8(((w0 >> 4) & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u), sc);
                            }
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                const uint32_t va[4] = {(&f[0][0].x)[b], (&f[1][0].x)[b], (&f[0][1].x)[b], (&f[1][1].x)[b]};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_16816(o[4 * w + b][nt], va, pt[u][nt][0], pt[u][nt][1]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) arrive(empty_bar + stage);
            }
            tiles_done += n;

            // ---- the eight warps' results as one: m and l first, then O, scaled, in two steps
            auto barrier = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); };
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[nt][e] += __shfl_xor_sync(full, l[nt][e], 4);
                    l[nt][e] += __shfl_xor_sync(full, l[nt][e], 8);
                    l[nt][e] += __shfl_xor_sync(full, l[nt][e], 16);
                    if (gr == 0) ml[warp][8 * nt + 2 * c + e] = make_float2(m[nt][e], l[nt][e]);
                }
            barrier();  // the segment before has been written out, too
            float M[NT][2], L[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float2 x[kWarps];
                    M[nt][e] = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        x[w] = ml[w][8 * nt + 2 * c + e];
                        if (x[w].y != 0.f) M[nt][e] = fmaxf(M[nt][e], x[w].x);  // (l is not 0: something was seen; NaN counts)
                    }
                    L[nt][e] = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        if (x[w].y != 0.f) L[nt][e] += exp2_approx(x[w].x - M[nt][e]) * x[w].y;
                    const float f = l[nt][e] != 0.f ? exp2_approx(m[nt][e] - M[nt][e]) : 0.f;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        // (of a row that the warp has seen nothing of, O is 0.  An f that underflows leaves a NaN of O one.)
                        o[j][nt][e] *= f;
                        o[j][nt][e + 2] *= f;
                    }
                }
            auto cell = [&](int w, int j, int nt) { return joined + ((w * (D / 16) + j) * NT + nt) * 128 + 4 * lane; };
            // group by group, each adds what the one after it has put down
#pragma unroll
            for (int z = C::kGroups - 1; z >= 0; --z) {
                if (group == z) {
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float4 *at = reinterpret_cast<float4 *>(cell(warp % C::kOfTile, j, nt));
                            float4 x = make_float4(o[j][nt][0], o[j][nt][1], o[j][nt][2], o[j][nt][3]);
                            if (z < C::kGroups - 1) x = make_float4(x.x + at->x, x.y + at->y, x.z + at->z, x.w + at->w);
                            *at = x;
                        }
                }
                if (z > 0) barrier();
            }
            const uint32_t bits = nf[seg & 1];  // (set before the barriers)
            if (tid == 0) nf[(seg + 1) & 1] = 0;
            barrier();

            // ---- out: warp w columns d = gr D / 8 + 4 w .. + 3 of rows 8 nt + 2 c + e
            const bool whole = g.starts && g.ends;
            const int slot = g.starts ? 1 : 0;
            float *part = a.parts + (size_t(blockIdx.x) * 2 + slot) * Cfg<D, true>::kPartFloats;
            if (!whole) {
                if (tid == 0) meta[slot] = make_int4(g.rows, g.ends, g.q.n0 + g.i0, g.h);
                if (slot) tail_part = true;
                else head_part = true;
            }
            if (warp < D / 32) {
                const int d = gr * (D / 8) + 4 * warp;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float4 v[2];  // by j: (d, row), (d, row + 1), (d + 1, row), (d + 1, row + 1)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int w = 0; w < C::kOfTile; ++w) {
                            const float4 x = *reinterpret_cast<const float4 *>(cell(w, 2 * warp + j, nt));
                            v[j] = make_float4(v[j].x + x.x, v[j].y + x.y, v[j].z + x.z, v[j].w + x.w);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * nt + 2 * c + e;
                        if (row >= g.rows) continue;
                        float out[4] = {e ? v[0].y : v[0].x, e ? v[0].w : v[0].z, e ? v[1].y : v[1].x, e ? v[1].w : v[1].z};
                        for (uint32_t b = bits; b; b &= b - 1) {
                            const int x = g.safe + __ffs(b) - 1;
                            if (!sees(nt, e, x)) continue;
                            const unsigned char *sc = scale_bytes<D>(a, g.s, g.h, x);
                            if (sc && (sc[d / 16] & 0x7f) == gdn::kNanScale) out[0] = out[1] = out[2] = out[3] = __uint_as_float(0x7fffffffu);
                        }
                        if (whole) {
                            const float inv = a.out / L[nt][e];
                            T *to = static_cast<T *>(a.o) +
                                    ((int64_t(g.q.n0) + g.i0 + row / a.G) * a.Hq + int64_t(g.h) * a.G + row % a.G) * D + d;
                            *reinterpret_cast<uint2 *>(to) = make_uint2(gdn::Half2<T>::pack(out[0] * inv, out[1] * inv),
                                                                        gdn::Half2<T>::pack(out[2] * inv, out[3] * inv));
                        } else {
                            if (warp == 0 && gr == 0) {
                                part[row] = M[nt][e];
                                part[kRows + row] = L[nt][e];
                            }
                            *reinterpret_cast<float4 *>(part + 2 * kRows + (size_t(d / 4) * kRows + row) * 4) =
                                make_float4(out[0], out[1], out[2], out[3]);
                        }
                    }
                }
            }
            ++seg;
        }
        if (tid == 0) {
            if (!head_part) meta[0] = make_int4(0, 0, 0, 0);
            if (!tail_part) meta[1] = make_int4(0, 0, 0, 0);
        }
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && abort_s) gdn::record_status(a.status, GDN_DEV_TIMEOUT);
}

template <typename T, int D, int NT>
int launch_few(const gdn_attn_dims *dims, att::Args a, int ctas, cudaStream_t st) {
    using C = Few<D, NT>;
    a.R = 8 * NT / a.G;
    auto k = kvq_few_kernel<T, D, NT>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem)) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    if (gdn::launch_pdl(k, dim3(unsigned(ctas)), dim3(C::kThreads), C::kSmem, st, a) != cudaSuccess) return GDN_ERR_LAUNCH;
    return launch_join<T, D, true>(dims, a, ctas, st);
}

template <typename T, int D>
int launch(const gdn_attn_dims *dims, att::Args a, void *workspace, int ctas, cudaStream_t st) {
    using C = att::Cfg<D, true>;
    a.meta = static_cast<int4 *>(workspace);
    a.parts = reinterpret_cast<float *>(a.meta + 2 * ctas);
    a.stall_ns = gdn::take_attention_stall(&a.stall_role);
    // Few rows (single tokens, 64 at d = 256 and 32 below, over up to 16,384 positions, 8 rows a head: 79 us at d = 256, 82-85 at
    // 128, 64 at 64; the other kernel 145, 228, 181.  16 rows: 110 at 128, 80 at 64; the other 230, 181, and at d = 256 146 for 168.)
    const int64_t rows = int64_t(a.G) * dims->max_seq_tokens;
    if (rows <= 8) return launch_few<T, D, 1>(dims, a, ctas, st);
    if constexpr (D < 256)
        if (rows <= 16) return launch_few<T, D, 2>(dims, a, ctas, st);
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
    if (!(scale * k_unit < 1.0e38f)) return GDN_ERR_ARG;  // (their product with log2(e) is a factor of the scores)
    bool empty = false;
    rc = check_attention(dims, q, q_stride, k_pool, v_pool, gdn::kv4_pool_bytes(dims), page_table, ctx_len, node_off, parents, scale, o,
                         workspace, workspace_size, gdn_attention_kvq_workspace_bytes(dims), status, &empty);
    if (rc || empty) return rc;
    const int ctas = gdn::sm_count_current();
    if (ctas < 1) return GDN_ERR_LAUNCH;
    const int64_t S = dims->n_seqs, N = dims->n_tokens, Hq = dims->h_q;
    const int G = int(Hq / dims->h_kv);
    // (rounded as fp32 rounds scale * log2(e), wherever the product with the unit lies)
    int e, e2, eu;
    const float mant = 2.f * std::frexp(std::frexp(scale, &e) * 1.4426950408889634f, &e2);
    std::frexp(k_unit, &eu);
    const int c_exp = e + e2 + eu - 2;
    att::Args a{q, q_stride, k_pool, v_pool, gdn::paged_layout(dims, page_table), ctx_len, node_off, parents,
                std::max(float(std::ldexp(double(mant), c_exp)), FLT_MIN), mant, c_exp, v_unit, o, status, nullptr, nullptr, int(S), int(N),
                dims->max_seq_tokens, int(Hq), dims->h_kv, G, att::kRows / G, 0, 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dims->dtype == GDN_BF16 ? launch_d<__nv_bfloat16>(dims, a, workspace, ctas, st)
                                   : launch_d<__half>(dims, a, workspace, ctas, st);
}
