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
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "gdn_attn.h"
#include "gdn_tma.h"

namespace {
namespace att {

constexpr int kRows = 128;
// m: log2 of the largest p when it is chosen, log2 of the p that moves it and, for D = 256, the sum of a tile's p
// that does.  A tile of equal scores right after a move sums to 64 2^kLift, below kMoveAtSum.
template <typename T> struct Reference {
    static constexpr float kLift = 0.f, kMoveAt = 8.f, kMoveAtSum = 16384.f;
};
template <> struct Reference<__half> {  // up to 65504
    static constexpr float kLift = 8.f, kMoveAt = 15.9f, kMoveAtSum = 61000.f;
};
constexpr int TK = 64;       // positions of a tile
// What an item costs beside its tiles (Q in, results out), in tiles.  Too little makes the CTAs with many
// short items the last (chunks of up to 701 tokens: 4 289 us, 8 263, 10 266; 64 trees 122.6, 119.5, 120.6),
// too much those with few long ones (64 single tokens: 186.9, 187.0, 187.2; 24 191.1).  Not measured for D = 64.
constexpr int kItemUnits = 10;
constexpr int kNfBufs = 16;  // the ring holds the values of 12 segments at most, and one may still be going out

template <int D_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr int kStreams = D == 256 ? 1 : 2;     // softmax warpgroups, each with an O of its own
    static constexpr int kRowWarps = 4 * kStreams;
    static constexpr int kTma = kRowWarps, kMmaS = kTma + 1, kMmaO = kTma + 2, kClean = kTma + 3;
    static constexpr int kThreads = 32 * (kRowWarps + 4);  // 8 or 12 warps: two or three to a scheduler
    static constexpr int kChunks = D / 64;                // 128-byte columns of a row
    static constexpr uint32_t kChunkBytes = TK * 128;
    static constexpr uint32_t kTile = TK * D * 2;         // 32, 16, 8 KB
    static constexpr int kStages = 196608 / kTile;
    static constexpr size_t kSmem = 1024 + 196608;
    // tensor-memory columns
    static constexpr int kSBufs = kStreams;
    static constexpr uint32_t kO = 0, kQ = kStreams * D, kS = kQ + D / 2, kP = kS + kSBufs * TK;
    static_assert(kP + 2 * (TK / 2) <= 512, "tensor memory");
    static __device__ __forceinline__ int s_buf(long long i) { return kSBufs == 2 ? int(i & 1) : 0; }
    static __device__ __forceinline__ uint32_t s_use(long long i) { return uint32_t(kSBufs == 2 ? i >> 1 : i); }
    static_assert(kStages / 2 + 2 <= kNfBufs, "flags of the segments in the ring");
    // place in the ring of a segment's K and V tile k of n: K_0 K_1 V_0 K_2 V_1 ... V_{n-1}
    static __device__ __forceinline__ int k_at(int k) { return k == 0 ? 0 : 2 * k - 1; }
    static __device__ __forceinline__ int v_at(int k, int n) { return k + 1 < n ? 2 * k + 2 : 2 * n - 1; }
    // workspace of a CTA: two parts (0: an item that began before, 1: one that goes on) of m, l and O
    static constexpr size_t kPartFloats = size_t(kRows) * (D + 2);
};

// A tile of keys or values lies as boxes of `rows` positions, each [64 columns][position]:
// pages of 16 and 32 tokens arrive as one box each.
__device__ __forceinline__ int box_rows(int shift) { return shift == 4 ? 16 : shift == 5 ? 32 : TK; }
template <typename C>
__device__ __forceinline__ uint32_t place(int rows, int r) {  // bytes from the tile's start to position r's first 64 columns
    const int box = r & ~(rows - 1);
    return uint32_t(box) * (128 * C::kChunks) + uint32_t(r - box) * 128;
}

struct Args {
    const void *__restrict__ q;
    int64_t q_stride;
    const void *__restrict__ v_pool;  // read directly only for values that are not finite
    gdn::PagedLayout pl;
    const int32_t *__restrict__ ctx_len, *__restrict__ node_off, *__restrict__ parents;
    float c;  // scale * log2(e)
    void *o;
    int32_t *status;
    float *parts;  // [CTA][2][part]
    int4 *meta;    // [CTA][2]: rows of the part (0: none), ends, token n0 + i0, key/value head
    int S, N, max_tokens, Hq, Hkv, G, R;  // R: tokens of a row tile
    uint64_t stall_ns;                    // test hook: a warp of CTA 0 waits for what never comes, so long (0: none)
    int stall_role;                       // 0 rows, 1 copies, 2 scores, 3 P V, 4 cleaning
};

// sum_{j < n} floor((a j + b) / m), a, b >= 0, m > 0: by Euclid's steps on (a, m)
__device__ __noinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
    long long r = 0;
    while (n > 0) {
        r += (a / m) * (n * (n - 1) / 2) + (b / m) * n;
        a %= m;
        b %= m;
        const long long y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const long long t = m;
        m = a;
        a = t;
    }
    return r;
}

// A sequence as the schedule sees it; n = 0 when it is empty or refused.
struct Seq {
    int n0, n, ctx;
};
struct RawSeq {
    int n0, n1, ctx;
};
__device__ __forceinline__ RawSeq load_raw(const Args &a, int s) { return {a.node_off[s], a.node_off[s + 1], a.ctx_len[s]}; }
__device__ __forceinline__ Seq checked(const Args &a, int s, const RawSeq &r, int *err = nullptr) {
    Seq q{r.n0, 0, r.ctx};
    const int n1 = r.n1;
    int e = 0;
    if (q.n0 < 0 || n1 < q.n0 || n1 > a.N || (s == 0 && q.n0 != 0) || (s == a.S - 1 && n1 != a.N) ||
        n1 - q.n0 > a.max_tokens)
        e = GDN_DEV_BAD_NODE_OFF;
    else if (q.ctx < 0 || int64_t(q.ctx) + (n1 - q.n0) > (int64_t(a.pl.width) << a.pl.shift))
        e = GDN_DEV_BAD_LEN;
    else
        q.n = n1 - q.n0;
    if (err) *err = e;
    return q;
}
// Units of work of row tile j: its tiles and kItemUnits at its front.
__device__ __forceinline__ int item_units(const Seq &q, int j, int R) {
    return (q.ctx + min((j + 1) * R, q.n) + TK - 1) / TK + kItemUnits;
}
// units of row tiles 0 .. j - 1 (j <= the number of row tiles - 1)
__device__ __forceinline__ long long units_before(const Seq &q, int j, int R) {
    return floor_sum(j, TK, R, (long long)q.ctx + R + TK - 1) + (long long)j * kItemUnits;
}
__device__ __forceinline__ long long head_units(const Seq &q, int R) {
    if (q.n == 0) return 0;
    const int J = (q.n + R - 1) / R;
    return units_before(q, J - 1, R) + item_units(q, J - 1, R);
}

struct Start {
    Seq q;
    int s, h, j, off;
    long long count;  // units of this CTA
};

// A CTA's run through its share, segment by segment (a segment: consecutive tiles
// of one item).  Every role walks it for itself.
struct Segment {
    int s, h, i0, rows, tile0, tile1;  // rows: valid rows of the tile
    bool starts, ends;
    int limit;  // positions of the item: ctx + tokens up to the tile's last
    int safe;   // positions below it are seen by every row
    Seq q;
};
struct Walk {
    const Args &a;
    int s, h, j, off;
    long long left;
    Seq q;
    RawSeq nx;  // of the next sequence, loaded one ahead and looked at when it is its turn
    __device__ Walk(const Args &a_, const Start &st) : a(a_), s(st.s), h(st.h), j(st.j), off(st.off), left(st.count) {
        q = st.q;
        if (left > 0 && s + 1 < a.S) nx = load_raw(a, s + 1);
    }
    __device__ __forceinline__ bool next(Segment &g) {
        while (left > 0) {
            const int total = item_units(q, j, a.R);
            const int take = int(min((long long)(total - off), left));
            g.s = s;
            g.h = h;
            g.i0 = j * a.R;
            const int toks = min(a.R, q.n - g.i0);
            g.rows = toks * a.G;
            g.tile0 = max(0, off - kItemUnits);
            g.tile1 = max(0, off + take - kItemUnits);
            g.starts = g.tile0 == 0;
            g.ends = off + take == total;
            g.limit = q.ctx + g.i0 + toks;
            g.safe = a.parents ? q.ctx : q.ctx + g.i0 + 1;
            g.q = q;
            left -= take;
            off += take;
            if (g.ends) {
                off = 0;
                if ((j + 1) * a.R >= q.n) {
                    j = 0;
                    if (++h == a.Hkv) {
                        h = 0;
                        while (left > 0 && s + 1 < a.S) {  // the next sequence with tokens
                            ++s;
                            q = checked(a, s, nx);
                            if (s + 1 < a.S) nx = load_raw(a, s + 1);
                            if (q.n > 0) break;
                        }
                    }
                } else {
                    ++j;
                }
            }
            if (g.tile1 > g.tile0) return true;  // (a share that ends in an item's front has no tile of it)
        }
        return false;
    }
};

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// D[tmem] (+)= A[tmem] x B[smem], 16-bit operands, fp32 accumulators
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// S = Q K^T of a tile that lies in boxes of kBox positions, box by box: products of N = 16 and 32 cost 9 and
// 16 cycles, in proportion to 64's 32, as long as their issue is straight-line code.
template <typename C, uint32_t kIdS, int kBox>
__device__ __forceinline__ void scores_of(uint32_t d, uint32_t q, uint32_t kb) {
    constexpr uint32_t id = kIdS ^ (uint32_t(TK >> 3) << 17) ^ (uint32_t(kBox >> 3) << 17);
#pragma unroll
    for (int r = 0; r < TK; r += kBox)
#pragma unroll
        for (int z = 0; z < C::D / 16; ++z)
            mma_f16_ta(d + r, q + 8 * z,
                       gdn::desc_sw128(kb) + uint64_t(r * 8 * C::kChunks + (z >> 2) * (kBox * 8) + 2 * (z & 3)), id, z > 0);
}
// MN-major operand in the 128-byte swizzle: 64 elements (128 bytes) of MN by 8 of K
// an atom; `lead` bytes from one atom of MN to the next, 1024 from one of K to the next.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t lead) {
    return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(lead >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int row, int chunk, int head, int page,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(chunk), "r"(head), "r"(page),
        "r"(gdn::smem_addr(bar))
        : "memory");
}
// Warp-collective: thread t writes 32 columns (words) of lane (taddr lane) + t.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(gdn::smem_addr(bar)) : "memory");
}
// Warp-collective bounded wait; false (for the whole warp) after a timeout anywhere in the CTA.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    bool ok = gdn::mbar_try_wait(bar, parity);
    if (!ok && !*abort_flag) ok = gdn::mbar_wait_bounded(bar, parity);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *abort_flag = 1;
    return ok;
}
// Two waits in one, where both are mostly over.
__device__ __forceinline__ bool wait_both(uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1, volatile int *abort_flag) {
    const bool ok = gdn::mbar_try_wait(b0, p0) & gdn::mbar_try_wait(b1, p1);
    if (__all_sync(0xffffffffu, ok)) return true;
    return wait_bar(b0, p0, abort_flag) && wait_bar(b1, p1, abort_flag);
}
// Which of the 32 positions from `base` on a row sees: all below `upto` (chain), or
// all below ctx and the bits of `line` from there (tree).
__device__ __forceinline__ uint32_t seen32(bool tree, int base, int ctx, int upto, unsigned long long line) {
    if (!tree) {
        const int n = upto - base;
        return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
    }
    const int rel = base - ctx;
    if (rel >= 0) return rel < 64 ? uint32_t(line >> rel) : 0u;
    if (rel <= -32) return 0xffffffffu;
    return uint32_t(line << -rel) | ((1u << -rel) - 1u);
}

}  // namespace att

template <typename T, int D>
__global__ void __launch_bounds__(att::Cfg<D>::kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                           const att::Args a) {
    using namespace att;
    using C = Cfg<D>;
    using Ref = Reference<T>;
    constexpr int kThreads = C::kThreads, kTma = C::kTma;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ uint64_t full_bar[C::kStages], empty_bar[C::kStages];
    __shared__ uint64_t s_bar[2], sfree_bar[2], p_bar[2], pv_bar[2], q_bar, ml_bar, ofree_bar, go_bar[2], clean_bar[2], drain_bar[2], never_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_s;
    __shared__ Start start_s;
    __shared__ long long wsum[kThreads / 32];
    __shared__ int tree_par[C::kRowWarps][gdn::kMaxSeqNodes];
    __shared__ float2 ml[2][C::kStreams][kRows];  // by segment: m and l of each stream's rows
    __shared__ uint32_t nf[kNfBufs][4];  // by segment: positions from `safe` on with values that are not finite
    volatile int *abort_flag = &abort_s;
    unsigned char *tiles =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t tb = gdn::smem_addr(tiles);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned full = 0xffffffffu;

    gdn::grid_dep_launch();
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            gdn::mbar_init(full_bar + i, 1);
            gdn::mbar_init(empty_bar + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            gdn::mbar_init(s_bar + i, 1);
            gdn::mbar_init(sfree_bar + i, 4);
            gdn::mbar_init(p_bar + i, 4);
            gdn::mbar_init(pv_bar + i, 1);
            gdn::mbar_init(go_bar + i, 1);
            gdn::mbar_init(clean_bar + i, 1);
            gdn::mbar_init(drain_bar + i, 1);
        }
        gdn::mbar_init(&q_bar, C::kRowWarps);
        gdn::mbar_init(&ml_bar, C::kRowWarps);
        gdn::mbar_init(&ofree_bar, C::kRowWarps);
        gdn::mbar_init(&never_bar, 1);
        gdn::fence_mbar_init();
        abort_s = 0;
        start_s.count = 0;
    }
    if (warp == C::kMmaS) {
        gdn::tmem_alloc(&tmem_slot, 512);
        gdn::tmem_relinquish();
    }
    gdn::grid_dep_wait();  // lengths, q, the pools and the workspace

    // ---- the schedule: units of all sequences, cut into equal shares ------------
    const int per = (a.S + kThreads - 1) / kThreads;
    long long mine = 0;
    Seq q0{0, 0, 0};  // the thread's first sequence (its only one up to kThreads of them)
    for (int k = 0; k < per; ++k) {
        const int s = tid * per + k;
        if (s >= a.S) break;
        int err;
        const Seq q = checked(a, s, load_raw(a, s), &err);
        if (k == 0) q0 = q;
        if (err && blockIdx.x == 0) gdn::record_status(a.status, err);
        mine += head_units(q, a.R) * a.Hkv;
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(full, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) wsum[warp] = inc;
    gdn::tc_fence_before_sync();
    __syncthreads();
    gdn::tc_fence_after_sync();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) before = total;
        total += wsum[w];
    }
    before += inc - mine;
    {
        const long long active = min((long long)gridDim.x, total);
        const int b = blockIdx.x;
        if (b < active) {
            // (32-bit division where it does: the 64-bit one is a call)
            const bool small = total < (1 << 23);  // times at most 2^8 CTAs and below 2^31
            const long long t0 = small && active <= 256 ? unsigned(total) * unsigned(b) / unsigned(active) : total * b / active;
            const long long t1 =
                small && active <= 256 ? unsigned(total) * unsigned(b + 1) / unsigned(active) : total * (b + 1) / active;
            if (mine > 0 && t0 >= before && t0 < before + mine) {  // one thread of the CTA
                long long x = t0 - before;
                for (int k = 0; k < per; ++k) {
                    const int s = tid * per + k;
                    const Seq q = k == 0 ? q0 : checked(a, s, load_raw(a, s));
                    const long long ht = head_units(q, a.R);
                    if (x >= ht * a.Hkv) {
                        x -= ht * a.Hkv;
                        continue;
                    }
                    const int h = small ? int(unsigned(x) / unsigned(ht)) : int(x / ht);
                    x -= h * ht;
                    int lo = 0, hi = (q.n + a.R - 1) / a.R;  // the last row tile with units_before <= x
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) / 2;
                        if (units_before(q, mid, a.R) <= x) lo = mid;
                        else hi = mid;
                    }
                    start_s = Start{q, s, h, lo, int(x - units_before(q, lo, a.R)), t1 - t0};
                    break;
                }
            }
        }
    }
    __syncthreads();
    const Start start = start_s;
    const uint32_t tmem = tmem_slot;
    Walk walk(a, start);
    Segment g;
    bool ok = true;  // this warp's; false once a wait has run out
    if (a.stall_ns && blockIdx.x == 0 && warp == (a.stall_role == 0 ? 0 : C::kRowWarps + a.stall_role - 1)) {
        ok = __all_sync(full, gdn::mbar_wait_bounded(&never_bar, 0, a.stall_ns));
        if (!ok) *abort_flag = 1;
    }

    if (warp == kTma) {
        // ---- keys and values by TMA -------------------------------------------------
        asm volatile("fence.proxy.async;" ::: "memory");  // what earlier kernels wrote, for the copies
        const int ps = 1 << a.pl.shift, np = max(1, TK / ps);  // pages of a tile
        // a box: the whole tile, a whole page (from 16 tokens on), or a page's 64 columns
        const bool pages = ps >= 16;
        const int bb = pages ? lane : lane / C::kChunks, bc = pages ? 0 : lane % C::kChunks;  // this lane's page, chunk
        const bool box_lane = bb < np;
        const uint32_t bytes = pages ? min(ps, TK) * 128u * C::kChunks : ps * 128u;
        const uint32_t dst = pages ? bb * bytes : bc * C::kChunkBytes + uint32_t(bb) * ps * 128u;
        // (Loads whose data are the first to leave L2, so that the parts stay there, gave 64 single tokens 185 for
        // 189 us and 64 trees 120 for 122, but where sequences share a prefix's pages, which no argument tells, cost
        // 306 for 291 us over 32,768 shared positions and 109 for 106 over 8,192.)
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;
        bool bad_page = false;
        auto load = [&](const CUtensorMap *map, int page, int row, int head) {
            if (!wait_bar(empty_bar + stage, phase ^ 1, abort_flag)) return false;
            const bool mine = box_lane && page >= 0;
            const unsigned m = __ballot_sync(full, mine);
            if (lane == 0) gdn::mbar_arrive_expect_tx(full_bar + stage, __popc(m) * bytes);
            __syncwarp();
            if (mine) tma_load_5d(tb + stage * C::kTile + dst, map, row, bc, head, page, full_bar + stage);
            ++issued;
            if (++stage == C::kStages) {
                stage = 0;
                phase ^= 1;
            }
            return true;
        };
        while (ok && walk.next(g)) {
            // the segment's page-table entries, 32 in each of two registers, loaded ahead and
            // looked at when their tile is requested
            const int32_t *table = a.pl.table + int64_t(g.s) * a.pl.width;
            const int last = (g.limit - 1) >> a.pl.shift;  // the item's last page
            int base = (g.tile0 * TK) >> a.pl.shift;
            auto entry = [&](int o) { return o <= last ? table[o] : -1; };
            int cur = entry(base + lane), nxt = entry(base + 32 + lane);
            auto page_of = [&](int first, int b) {  // page `first + b` (checked)
                const int o = first + b - base;
                const int lo = __shfl_sync(full, cur, o & 31), hi = __shfl_sync(full, nxt, o & 31);
                const int p = o < 32 ? lo : hi;
                if (first + b > last) return -1;
                if (p < 0 || p >= a.pl.n_pages) {
                    bad_page = true;
                    return -1;
                }
                return p;
            };
            int v_page = -1;
            for (int t = g.tile0; t <= g.tile1 && ok; ++t) {
                int page = -1;
                if (t < g.tile1) {
                    const int first = (t * TK) >> a.pl.shift;
                    if (first - base >= 32) {
                        cur = nxt;
                        base += 32;
                        nxt = entry(base + 32 + lane);
                    }
                    page = page_of(first, box_lane ? bb : 0);
                    ok = load(&kmap, page, (t * TK) & (ps - 1), g.h);
                }
                if (ok && t > g.tile0) ok = load(&vmap, v_page, ((t - 1) * TK) & (ps - 1), g.h);
                v_page = page;
            }
        }
        if (bad_page) gdn::record_status(a.status, GDN_DEV_BAD_PAGE);
        // The last copies into each stage are waited for (bounded) whatever has happened: when a role that was to
        // take them has given up, this warp may have requested its last one all the same, and the CTA must not
        // leave with copies under way into its shared memory.
        const int n = int(min(issued, (long long)C::kStages));
        for (int k = 0; k < n; ++k) {
            if (stage == 0) {
                stage = C::kStages;
                phase ^= 1;
            }
            --stage;
            gdn::mbar_wait_bounded(full_bar + stage, phase);
        }
    } else if (warp == C::kMmaS || warp == C::kMmaO) {
        // ---- the products: one warp issues S = Q K^T, one O += P V, so that neither's
        //      waits keep the tensor cores from the other's work -------------------------
        constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
        constexpr uint32_t kIdS = (1u << 4) | (fmt << 7) | (fmt << 10) | (uint32_t(TK >> 3) << 17) | (8u << 24);
        constexpr uint32_t kIdO = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 16) | (uint32_t(D >> 3) << 17) | (8u << 24);
        const bool is_s = warp == C::kMmaS;
        const int rows = box_rows(a.pl.shift);
        uint32_t seg = 0, masked = 0, asked = 0;
        long long loads = 0, tile = 0;  // of the segments before: ring places, tiles (buffers and phases of S, P)
        while (ok && walk.next(g)) {
            const int n = g.tile1 - g.tile0;
            if (is_s) {
                ok = wait_bar(&q_bar, seg & 1, abort_flag);
                for (int k = 0; k < n && ok; ++k) {
                    const long long at = loads + C::k_at(k), i = tile + k;
                    const int stage = int(at % C::kStages);
                    ok = wait_bar(full_bar + stage, uint32_t(at / C::kStages) & 1, abort_flag);
                    const int sb = C::s_buf(i);  // its last scores have been read
                    if (i >= C::kSBufs) ok = ok && wait_bar(sfree_bar + sb, (C::s_use(i) - 1) & 1, abort_flag);
                    if (!ok) break;
                    gdn::tc_fence_after_sync();
                    if (elect_one()) {
                        const uint32_t kb = tb + stage * C::kTile, d = tmem + C::kS + uint32_t(sb) * TK;
                        if (rows == 64) scores_of<C, kIdS, 64>(d, tmem + C::kQ, kb);
                        else if (rows == 32) scores_of<C, kIdS, 32>(d, tmem + C::kQ, kb);
                        else scores_of<C, kIdS, 16>(d, tmem + C::kQ, kb);
                        gdn::mma_commit(s_bar + sb);
                        gdn::mma_commit(empty_bar + stage);
                    }
                    __syncwarp();
                }
            } else {
                for (int k = 0; k < n && ok; ++k) {
                    const long long at = loads + C::v_at(k, n), i = tile + k;
                    const int stage = int(at % C::kStages);
                    ok = wait_bar(full_bar + stage, uint32_t(at / C::kStages) & 1, abort_flag);
                    if (!ok) break;
                    // cleaning runs beside the softmax: this tile's is asked for now, the next one's too if its
                    // values are there (two barriers each, as one may be under way while another is asked for)
                    const bool clean = (g.tile0 + k + 1) * TK > g.safe;
                    if (clean && asked == masked) {
                        if (lane == 0) arrive(go_bar + (asked & 1));
                        ++asked;
                    }
                    if (k + 1 < n && (g.tile0 + k + 2) * TK > g.safe) {
                        const long long nx = loads + C::v_at(k + 1, n);
                        if (__all_sync(full, gdn::mbar_test_wait(full_bar + nx % C::kStages, uint32_t(nx / C::kStages) & 1))) {
                            if (lane == 0) arrive(go_bar + (asked & 1));
                            ++asked;
                        }
                    }
                    ok = wait_bar(p_bar + (i & 1), uint32_t(i >> 1) & 1, abort_flag);
                    // both warpgroups read both O at a segment's end (one alone is done before it makes this P)
                    if (C::kStreams == 2 && k == 0 && seg > 0) ok = ok && wait_bar(&ofree_bar, (seg - 1) & 1, abort_flag);
                    if (clean) {
                        ok = ok && wait_bar(clean_bar + (masked & 1), (masked >> 1) & 1, abort_flag);
                        ++masked;
                    }
                    if (!ok) break;
                    gdn::tc_fence_after_sync();
                    if (elect_one()) {
                        const uint32_t vb = tb + stage * C::kTile, p = tmem + C::kP + uint32_t(i & 1) * (TK / 2);
                        const uint32_t o = tmem + C::kO + (C::kStreams == 2 ? uint32_t(i & 1) * D : 0u);
#pragma unroll
                        for (int z = 0; z < TK / 16; ++z)
                            mma_f16_ta(o, p + 8 * z, desc_mn_sw128(vb + place<C>(rows, 16 * z), rows * 128), kIdO,
                                       z > 0 || k >= C::kStreams);
                        gdn::mma_commit(pv_bar + (i & 1));
                        gdn::mma_commit(empty_bar + stage);
                    }
                    __syncwarp();
                }
            }
            loads += 2 * n;
            tile += n;
            ++seg;
        }
        if (elect_one()) gdn::mma_commit(drain_bar + (is_s ? 0 : 1));
        __syncwarp();
        gdn::mbar_wait_bounded(drain_bar + (is_s ? 0 : 1), 0);
    } else if (warp == C::kClean) {
        // ---- values of tiles that not every row sees whole ----------------------------
        long long loads = 0;  // ring position of the segment's first load
        uint32_t seg = 0, masked = 0;
        // the exponents of two values, and their lowest bits
        constexpr uint32_t kExp2 = std::is_same<T, __nv_bfloat16>::value ? 0x7F807F80u : 0x7C007C00u;
        constexpr uint32_t kLow2 = std::is_same<T, __nv_bfloat16>::value ? 0x00800080u : 0x04000400u;
        const int rows = box_rows(a.pl.shift);
        while (ok && walk.next(g)) {
            const int n = g.tile1 - g.tile0;
            // this warp is the first to come to a segment: its Q rows are on their way into L2 while the last
            // segment's results go out
            for (int u = lane; u < g.rows * C::kChunks; u += 32) {
                const int r = u / C::kChunks;
                const T *src = static_cast<const T *>(a.q) + (int64_t(g.q.n0) + g.i0 + r / a.G) * a.q_stride +
                               (int64_t(g.h) * a.G + r % a.G) * D + 64 * (u % C::kChunks);
                asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
            }
            uint32_t bits[4] = {0, 0, 0, 0};
            for (int t = max(g.tile0, g.safe / TK); t < g.tile1 && ok; ++t) {
                const long long at = loads + C::v_at(t - g.tile0, n);
                const int stage = int(at % C::kStages);
                const uint32_t mk = masked++;
                ok = wait_bar(go_bar + (mk & 1), (mk >> 1) & 1, abort_flag) &&
                     wait_bar(full_bar + stage, uint32_t(at / C::kStages) & 1, abort_flag);
                if (!ok) break;
                const int r0 = max(0, g.safe - t * TK);  // rows (positions) that some rows do not see
                unsigned char *vt = tiles + size_t(stage) * C::kTile;
                constexpr int kRowPieces = C::kChunks * 8, kStep = 32;  // 16-byte pieces
                auto piece = [&](int u) {
                    const int r = r0 + u / kRowPieces, c16 = u % kRowPieces;
                    return reinterpret_cast<uint4 *>(vt + place<C>(rows, r) + (c16 >> 3) * (rows * 128) +
                                                     (c16 & 7) * 16);
                };
                const int some = min(max(g.limit - t * TK - r0, 0), TK - r0) * kRowPieces;  // seen by some rows
                for (int u0 = lane; u0 < some; u0 += 8 * kStep) {
                    uint4 v[8];
                    uint32_t any = 0;  // the top bit of a half is set where its exponent is all ones
#pragma unroll
                    for (int z = 0; z < 8; ++z) v[z] = *piece(min(u0 + z * kStep, some - 1));
#pragma unroll
                    for (int z = 0; z < 8; ++z)
                        any |= (((v[z].x & kExp2) + kLow2) | ((v[z].y & kExp2) + kLow2) | ((v[z].z & kExp2) + kLow2) |
                                ((v[z].w & kExp2) + kLow2)) & 0x80008000u;
                    if (any == 0) continue;
#pragma unroll 1
                    for (int z = 0; z < 8; ++z) {
                        const int u = u0 + z * kStep;
                        if (u >= some) break;
                        uint32_t *e = reinterpret_cast<uint32_t *>(piece(u));
                        bool odd = false;
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t x = e[i], f = ((x & kExp2) + kLow2) & 0x80008000u;
                            if (f) {
                                e[i] = x & ~((f & 0x80000000u ? 0xFFFF0000u : 0u) | (f & 0x8000u ? 0xFFFFu : 0u));
                                odd = true;
                            }
                        }
                        if (odd) {
                            const int bit = t * TK + r0 + u / kRowPieces - g.safe;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (i == bit >> 5) bits[i] |= 1u << (bit & 31);
                        }
                    }
                }
                for (int u = some + lane; u < (TK - r0) * kRowPieces; u += kStep) *piece(u) = make_uint4(0, 0, 0, 0);
                gdn::fence_proxy_async_smem();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    bits[i] = __reduce_or_sync(full, bits[i]);
                    if (lane == i) nf[seg % kNfBufs][i] = bits[i];
                }
                __syncwarp();
                if (lane == 0) arrive(clean_bar + (mk & 1));
            }
            loads += 2 * n;
            ++seg;
        }
    } else {
        // ---- rows ------------------------------------------------------------------------
        const int w = warp & 3, stream = warp >> 2;        // lanes 32 w .. of tensor memory; the warpgroup
        const uint32_t trow = tmem + (uint32_t(w) << 21);  // this warp's lanes
        const int row = 32 * w + lane;
        constexpr int kCols = D / C::kStreams;             // columns of Q and of the results that a warpgroup moves
        const int col0 = stream * kCols;
        long long tile = 0;  // tiles of the segments before
        uint32_t seg = 0;
        const float c = a.c;
        int4 *meta = a.meta + 2 * blockIdx.x;
        bool head_part = false, tail_part = false;
        int line_s = -1;
        // A segment's Q rows into tensor memory, once every S of the segment before has been formed.
        auto load_q = [&](const Segment &sg) {
            if (w * 32 < sg.rows) {
                const int hd = sg.h * a.G + row % a.G;
                const bool live = row < sg.rows;
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) +
                                                                   (int64_t(sg.q.n0) + sg.i0 + row / a.G) * a.q_stride + int64_t(hd) * D);
                constexpr int kAhead = C::kStreams == 2 ? 1 : 2;  // chunks whose loads go out before the first is waited for
#pragma unroll
                for (int z0 = 0; z0 < (C::kChunks + C::kStreams - 1) / C::kStreams; z0 += kAhead) {
                    uint32_t q[kAhead][32];
#pragma unroll
                    for (int z = 0; z < kAhead; ++z) {
                        const int cc = (z0 + z) * C::kStreams + (C::kStreams == 2 ? stream : 0);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint4 v = live && cc < C::kChunks ? src[8 * cc + k] : make_uint4(0, 0, 0, 0);
                            q[z][4 * k] = v.x;
                            q[z][4 * k + 1] = v.y;
                            q[z][4 * k + 2] = v.z;
                            q[z][4 * k + 3] = v.w;
                        }
                    }
                    __syncwarp();  // lanes without a row have loaded nothing; the stores are the whole warp's
#pragma unroll
                    for (int z = 0; z < kAhead; ++z) {
                        const int cc = (z0 + z) * C::kStreams + (C::kStreams == 2 ? stream : 0);
                        if (cc < C::kChunks) tmem_st32(trow + C::kQ + 32 * cc, q[z]);
                    }
                }
                tmem_wait_st();
            }
            gdn::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive(&q_bar);
        };
        bool more = ok && walk.next(g);
        if (more) load_q(g);
        while (ok && more) {
            const int n = g.tile1 - g.tile0;
            const bool live_warp = w * 32 < g.rows, live = row < g.rows;
            const int i = g.i0 + row / a.G, hd = g.h * a.G + row % a.G;
            // the row's ancestors
            unsigned long long line = 0;
            if (a.parents && live_warp) {
                if (line_s != g.s) {
                    __syncwarp();
                    for (int x = lane; x < g.q.n; x += 32) tree_par[warp][x] = a.parents[g.q.n0 + x];
                    __syncwarp();
                    line_s = g.s;
                }
                if (live) {
                    for (int x = i; x >= 0;) {
                        line |= 1ull << x;
                        const int p = tree_par[warp][x];
                        if (p >= x || p < -1) {
                            gdn::record_status(a.status, GDN_DEV_BAD_PARENT);
                            break;
                        }
                        x = p;
                    }
                }
                __syncwarp();
            }
            const int upto = g.q.ctx + i + 1;
            float m = -INFINITY, l = 0.f;
            int done = 0;  // tiles of this warpgroup in this segment
            for (int k = C::kStreams == 2 ? int((tile ^ stream) & 1) : 0; k < n; k += C::kStreams, ++done) {
                const long long it = tile + k;
                const int t = g.tile0 + k, buf = int(it & 1), sb = C::s_buf(it);
                // With one stream the place of P is awaited here too (the product of two tiles before has read
                // it, and the wait is over as a rule); with two it is this warpgroup's last product's.
                if (C::kStreams == 1 && it >= 2)
                    ok = wait_both(s_bar + sb, C::s_use(it) & 1, pv_bar + buf, uint32_t((it >> 1) - 1) & 1, abort_flag);
                else
                    ok = wait_bar(s_bar + sb, C::s_use(it) & 1, abort_flag);
                if (!ok) break;
                float sv[2][32];
                if (live_warp) {
                    gdn::tc_fence_after_sync();
                    const uint32_t ts = trow + C::kS + uint32_t(sb) * TK;
                    gdn::tmem_ld32x2(ts, ts + 32, sv[0], sv[1]);
                    gdn::tc_fence_before_sync();
                }
                __syncwarp();
                if (lane == 0) arrive(sfree_bar + sb);
                if (live_warp) {
                    if ((t + 1) * TK > g.safe) {
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t vis = seen32(a.parents != nullptr, t * TK + 32 * z, g.q.ctx, upto, line);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((vis >> e) & 1)) sv[z][e] = -INFINITY;
                        }
                    }
                    auto tile_max = [&] {
                        float mv[8];  // eight chains: few warps share a scheduler, so latency counts
#pragma unroll
                        for (int e = 0; e < 8; ++e) mv[e] = -INFINITY;
#pragma unroll
                        for (int z = 0; z < 2; ++z)
#pragma unroll
                            for (int e = 0; e < 32; ++e) mv[e & 7] = fmaxf(mv[e & 7], sv[z][e]);
                        return c * fmaxf(fmaxf(fmaxf(mv[0], mv[1]), fmaxf(mv[2], mv[3])),
                                         fmaxf(fmaxf(mv[4], mv[5]), fmaxf(mv[6], mv[7])));
                    };
                    uint32_t r[32];
                    auto weights = [&] {  // P of the tile; its sum
                        const float mu = m == -INFINITY ? 0.f : m;  // a row that has seen nothing yet
                        const uint64_t c2 = gdn::f2pack(c, c), mu2 = gdn::f2pack(-mu, -mu);
                        uint64_t sum[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[e] = gdn::f2pack(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float *x = &sv[e >> 4][2 * (e & 15)];
                            const float2 y = gdn::f2unpack(gdn::fma2(gdn::f2pack(x[0], x[1]), c2, mu2));
                            const float p0 = exp2_approx(y.x), p1 = exp2_approx(y.y);
                            sum[e & 3] = gdn::add2(sum[e & 3], gdn::f2pack(p0, p1));
                            r[e] = gdn::Half2<T>::pack(p0, p1);
                        }
                        const float2 s2 = gdn::f2unpack(gdn::add2(gdn::add2(sum[0], sum[1]), gdn::add2(sum[2], sum[3])));
                        return s2.x + s2.y;
                    };
                    // m moves to what the tile's maximum asks for where `move` says so; O may be scaled once this
                    // warpgroup's product before this one has added to it
                    auto move_to = [&](float mx, bool move) {
                        const float f = move ? exp2_approx(m - (mx - Ref::kLift)) : 1.f;
                        if (move) m = mx - Ref::kLift;
                        l *= f;
                        if (done == 0) return true;
                        const long long pr = it - C::kStreams;
                        if (!wait_bar(pv_bar + (pr & 1), uint32_t(pr >> 1) & 1, abort_flag)) return false;
                        gdn::tc_fence_after_sync();
#pragma unroll 1
                        for (int cc = 0; cc < D; cc += 32) {
                            float v[32];
                            uint32_t o[32];
                            gdn::tmem_ld32(trow + C::kO + stream * D + cc, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(v[e] * f);
                            tmem_st32(trow + C::kO + stream * D + cc, o);
                        }
                        return true;
                    };
                    if (C::kStreams == 2) {
                        const float mx = tile_max();
                        if (m == -INFINITY) m = mx - Ref::kLift;
                        const bool move = mx > m + Ref::kMoveAt;
                        if (__any_sync(full, move)) ok = move_to(mx, move);
                        if (!ok) break;
                        l += weights();
                    } else {
                        if (__any_sync(full, m == -INFINITY)) {  // the first positions that the row sees
                            const float mx = tile_max();
                            if (m == -INFINITY) m = mx - Ref::kLift;
                        }
                        float sum = weights();
                        const bool move = sum > Ref::kMoveAtSum;
                        if (__any_sync(full, move)) {
                            ok = move_to(tile_max(), move);
                            if (!ok) break;
                            sum = weights();
                        }
                        l += sum;
                    }
                    // the place of P: the product of two tiles before has read it
                    if (C::kStreams == 2 && it >= 2) {
                        ok = wait_bar(pv_bar + buf, uint32_t((it >> 1) - 1) & 1, abort_flag);
                        if (!ok) break;
                        gdn::tc_fence_after_sync();
                    }
                    tmem_st32(trow + C::kP + uint32_t(buf) * (TK / 2), r);
                    tmem_wait_st();
                    gdn::tc_fence_before_sync();
                } else if (C::kStreams == 2 && it >= 2) {  // in step with the others, so that no phase is passed twice
                    ok = wait_bar(pv_bar + buf, uint32_t((it >> 1) - 1) & 1, abort_flag);
                    if (!ok) break;
                }
                __syncwarp();
                if (lane == 0) arrive(p_bar + buf);
            }
            if (!ok) break;
            // ---- the next segment's Q in, so that its first scores are formed meanwhile -------
            if (C::kStreams == 2) {  // the last S may be the other warpgroup's
                const long long it = tile + n - 1;
                ok = wait_bar(s_bar + C::s_buf(it), C::s_use(it) & 1, abort_flag);
                if (!ok) break;
            }
            Segment next;
            more = walk.next(next);
            if (more) load_q(next);
            // ---- the segment's rows out ---------------------------------------------------
            if (done > 0) {  // this warpgroup's last product (all before it are complete with it)
                const long long it = tile + n - 1 - (C::kStreams == 2 ? int((tile + n - 1 - stream) & 1) : 0);
                ok = wait_bar(pv_bar + (it & 1), uint32_t(it >> 1) & 1, abort_flag);
                if (!ok) break;
            }
            float f0 = 1.f, f1 = 0.f;  // factors of the streams' O
            bool s0 = true, s1 = false;  // whether the streams have seen anything (l is not 0: NaN counts, and stays)
            if (C::kStreams == 2) {
                ml[seg & 1][stream][row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) arrive(&ml_bar);
                ok = wait_bar(&ml_bar, seg & 1, abort_flag);
                if (!ok) break;
                const float2 x0 = ml[seg & 1][0][row], x1 = ml[seg & 1][C::kStreams - 1][row];
                m = fmaxf(x0.x, x1.x);
                // (the O of a stream that has seen nothing may never have been written)
                s0 = x0.y != 0.f;
                s1 = x1.y != 0.f;
                f0 = exp2_approx(x0.x - m);
                f1 = exp2_approx(x1.x - m);
                l = (s0 ? f0 * x0.y : 0.f) + (s1 ? f1 * x1.y : 0.f);
            }
            gdn::tc_fence_after_sync();
            const bool whole = g.starts && g.ends;
            const int slot = g.starts ? 1 : 0;
            float *part = a.parts + (size_t(blockIdx.x) * 2 + slot) * C::kPartFloats;
            if (!whole) {
                if (tid == 0) meta[slot] = make_int4(g.rows, g.ends, g.q.n0 + g.i0, g.h);
                if (slot) tail_part = true;
                else head_part = true;
                if (live && stream == 0) {
                    part[row] = m;
                    part[kRows + row] = l;
                }
            }
            uint32_t bits[4] = {0, 0, 0, 0};
            bool odd = false;
            if (g.tile1 * TK > g.safe) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bits[k] = *reinterpret_cast<volatile uint32_t *>(&nf[seg % kNfBufs][k]);
                    odd |= bits[k] != 0;
                }
            }
            const float inv = 1.f / l;
            if (live_warp) {
                T *orow = static_cast<T *>(a.o) + ((int64_t(g.q.n0) + i) * a.Hq + hd) * D;
#pragma unroll 1
                for (int cc = col0; cc < col0 + kCols; cc += 32) {
                    float v[32];
                    // rows past the last and rows with other non-finite values have gone other ways; the loads
                    // from tensor memory are the whole warp's, together
                    __syncwarp();
                    if (C::kStreams == 2) {
                        float v1[32];
                        gdn::tmem_ld32x2(trow + C::kO + cc, trow + C::kO + D + cc, v, v1);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[e] = (s0 ? f0 * v[e] : 0.f) + (s1 ? f1 * v1[e] : 0.f);
                    } else {
                        gdn::tmem_ld32(trow + C::kO + cc, v);
                    }
                    if (odd && live) {  // values that are not finite, for the rows that see them
                        for (int k = 0; k < 4; ++k)
                            for (uint32_t b = bits[k]; b; b &= b - 1) {
                                const int x = g.safe + 32 * k + __ffs(b) - 1;
                                if (!(seen32(a.parents != nullptr, x, g.q.ctx, upto, line) & 1)) continue;
                                const int64_t at = gdn::position_offset(a.pl, g.s, x);
                                if (at < 0) continue;
                                const T *vr = static_cast<const T *>(a.v_pool) + at + int64_t(g.h) * a.pl.head_stride + cc;
                                for (int e = 0; e < 32; ++e) {
                                    const float y = float(vr[e]);
                                    if (!(fabsf(y) < INFINITY)) {
#pragma unroll
                                        for (int z = 0; z < 32; ++z)
                                            if (z == e) v[z] += y;
                                    }
                                }
                            }
                    }
                    if (live && whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float y[8];
#pragma unroll
                            for (int z = 0; z < 8; ++z) y[z] = v[e + z] * inv;
                            *reinterpret_cast<uint4 *>(orow + cc + e) = gdn::pack8<T>(y);
                        }
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)  // column group, then row: neighbours side by side
                            *reinterpret_cast<float4 *>(part + 2 * kRows + (size_t((cc + e) / 4) * kRows + row) * 4) =
                                make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                }
            }
            if (C::kStreams == 2) {
                gdn::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive(&ofree_bar);
            }
            tile += n;
            ++seg;
            g = next;
        }
        if (tid == 0) {
            if (!head_part) meta[0] = make_int4(0, 0, 0, 0);
            if (!tail_part) meta[1] = make_int4(0, 0, 0, 0);
        }
    }
    __syncwarp();  // lanes may come from bounded waits of their own
    gdn::tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && abort_s) gdn::record_status(a.status, GDN_DEV_TIMEOUT);
    if (warp == C::kMmaS) gdn::tmem_dealloc(tmem, 512);
}

// Joins the parts of items that more than one CTA worked on: block (b, y) takes its
// share of the item that begins in CTA b and goes on in b + 1, ...  A unit is four
// columns of a row.  Few parts: a thread takes a unit and all its parts.  Many (one
// long sequence spread over the GPU): the block's warps take the parts in turn for 32
// units at a time and their eight sums are joined in order.  Bound by latency; every
// thread has the loads of four parts under way (one at a time took 24 us for 126 parts).
struct Joined {
    float m, l;
    float4 o;
};
__device__ __forceinline__ void join(Joined &a, const Joined &b) {
    if (b.l == 0.f) return;  // nothing seen in that part (l is NaN where a score is)
    if (a.l == 0.f) {
        a = b;
        return;
    }
    const float M = fmaxf(a.m, b.m), f = att::exp2_approx(a.m - M), w = att::exp2_approx(b.m - M);
    a.m = M;
    a.l = fmaf(w, b.l, f * a.l);
    a.o.x = fmaf(w, b.o.x, f * a.o.x);
    a.o.y = fmaf(w, b.o.y, f * a.o.y);
    a.o.z = fmaf(w, b.o.z, f * a.o.z);
    a.o.w = fmaf(w, b.o.w, f * a.o.w);
}

template <typename T, int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const att::Args a, int ctas) {
    using C = att::Cfg<D>;
    __shared__ Joined sums[8][32];
    gdn::grid_dep_launch();
    gdn::grid_dep_wait();
    const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int4 me = a.meta[2 * b + 1];
    if (me.x <= 0 || me.x > att::kRows) return;
    int last = ctas;  // the CTA with the item's end, looked for 32 at a time
    for (int k0 = b + 1; k0 < ctas && last == ctas; k0 += 32) {
        const int k = k0 + lane;
        bool end = k == ctas - 1;
        if (k < ctas) {
            const int4 m = a.meta[2 * k];
            end |= m.x <= 0 || m.y != 0;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, end);
        if (hit) last = k0 + __ffs(hit) - 1;
    }
    if (last >= ctas) return;
    const int rows = me.x, units = rows * (D / 4), parts = last - b + 1;
    // unit u over parts b + k0, b + k0 + step, ...
    auto gather = [&](int u, int k0, int step) {
        const int row = u % rows, c4 = u / rows;
        Joined acc{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        for (int k = k0; k < parts; k += 4 * step) {
            Joined p[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int kk = min(k + z * step, parts - 1) + b;
                const float *part = a.parts + (size_t(kk) * 2 + (kk == b)) * C::kPartFloats;
                p[z].m = part[row];
                p[z].l = part[att::kRows + row];
                p[z].o = *reinterpret_cast<const float4 *>(part + 2 * att::kRows + (size_t(c4) * att::kRows + row) * 4);
            }
#pragma unroll
            for (int z = 0; z < 4; ++z)
                if (k + z * step < parts) join(acc, p[z]);
        }
        return acc;
    };
    auto store = [&](int u, const Joined &r) {
        const int row = u % rows, c4 = u / rows;
        const float inv = 1.f / r.l;
        T *out = static_cast<T *>(a.o) + ((int64_t(me.z) + row / a.G) * a.Hq + me.w * a.G + row % a.G) * D + 4 * c4;
        *reinterpret_cast<uint2 *>(out) = make_uint2(gdn::Half2<T>::pack(r.o.x * inv, r.o.y * inv),
                                                     gdn::Half2<T>::pack(r.o.z * inv, r.o.w * inv));
    };
    if (parts <= 4) {
        for (int u = blockIdx.y * 256 + threadIdx.x; u < units; u += gridDim.y * 256) store(u, gather(u, 0, 1));
        return;
    }
    for (int u0 = blockIdx.y * 32; u0 < units; u0 += gridDim.y * 32) {
        const int u = u0 + lane;
        sums[warp][lane] = gather(min(u, units - 1), warp, 8);
        __syncthreads();
        if (warp == 0 && u < units) {
            Joined r = sums[0][lane];
#pragma unroll
            for (int w = 1; w < 8; ++w) join(r, sums[w][lane]);
            store(u, r);
        }
        __syncthreads();
    }
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

size_t workspace_bytes(const gdn_attn_dims *dims, int ctas) {
    return size_t(ctas) * (2 * att::kRows * size_t(dims->d_head + 2) * 4 + 2 * sizeof(int4));
}

std::atomic<uint64_t> g_stall{0};  // the pending test stall: role in the top byte, ns below

template <typename T, int D>
int launch(const gdn_attn_dims *dims, const void *k_pool, att::Args a, void *workspace, int ctas, cudaStream_t st) {
    using C = att::Cfg<D>;
    CUtensorMap kmap, vmap;
    const int ps = dims->page_size;
    const uint32_t rows = uint32_t(ps < att::TK ? ps : att::TK);
    int rc;
    const uint32_t chunks = ps >= 16 ? C::kChunks : 1;
    if ((rc = encode_kv_pages(&kmap, k_pool, dims, rows, chunks)) ||
        (rc = encode_kv_pages(&vmap, a.v_pool, dims, rows, chunks)))
        return rc;
    a.meta = static_cast<int4 *>(workspace);
    a.parts = reinterpret_cast<float *>(a.meta + 2 * ctas);
    const uint64_t stall = g_stall.exchange(0);
    a.stall_ns = stall & ((uint64_t(1) << 56) - 1);
    a.stall_role = int(stall >> 56);
    auto k = paged_attention_kernel<T, D>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem)) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    if (gdn::launch_pdl(k, dim3(unsigned(ctas)), dim3(C::kThreads), C::kSmem, st, kmap, vmap, a) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    const int units = a.G * (dims->max_seq_tokens < a.R ? dims->max_seq_tokens : a.R) * (D / 4);  // of a part, at most
    const unsigned y = units >= 16 * 32 ? 16 : unsigned(units + 31) / 32;
    return gdn::launch_pdl(attention_join_kernel<T, D>, dim3(unsigned(ctas), y), dim3(256), 0, st, a, ctas) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_LAUNCH;
}

template <typename T>
int launch_d(const gdn_attn_dims *dims, const void *k_pool, const att::Args &a, void *workspace, int ctas,
             cudaStream_t st) {
    switch (dims->d_head) {
        case 64: return launch<T, 64>(dims, k_pool, a, workspace, ctas, st);
        case 128: return launch<T, 128>(dims, k_pool, a, workspace, ctas, st);
        default: return launch<T, 256>(dims, k_pool, a, workspace, ctas, st);
    }
}

}  // namespace

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
    if (!status) return GDN_ERR_NULL;
    if (parents && dims->max_seq_tokens > gdn::kMaxSeqNodes) return GDN_ERR_DIMS;
    if (!(scale > 0.0f) || !(scale < 3.0e38f)) return GDN_ERR_ARG;
    const int64_t S = dims->n_seqs, N = dims->n_tokens, Hq = dims->h_q, D = dims->d_head;
    if (S == 0 || N == 0) return GDN_OK;
    if (!q || !k_pool || !v_pool || !page_table || !ctx_len || !node_off || !o || !workspace) return GDN_ERR_NULL;
    const size_t need = gdn_attention_workspace_bytes(dims);
    if (workspace_size < 0 || size_t(workspace_size) < need) return GDN_ERR_ARG;
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
    const int ctas = gdn::sm_count_current();
    if (ctas < 1) return GDN_ERR_LAUNCH;
    const int G = int(Hq / dims->h_kv);
    att::Args a{q, q_stride, v_pool, gdn::paged_layout(dims, page_table), ctx_len, node_off, parents,
                scale * 1.4426950408889634f, o, status, nullptr, nullptr, int(S), int(N), dims->max_seq_tokens, int(Hq),
                dims->h_kv, G, att::kRows / G, 0, 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dims->dtype == GDN_BF16 ? launch_d<__nv_bfloat16>(dims, k_pool, a, workspace, ctas, st)
                                   : launch_d<__half>(dims, k_pool, a, workspace, ctas, st);
}

extern "C" void gdn_test_stall_next_attention(uint64_t wait_ns, int role) {
    if (role < 0 || role > 4) return;
    g_stall.store(std::min<uint64_t>(wait_ns, gdn::kWaitLimitNs) | (uint64_t(role) << 56));
}
