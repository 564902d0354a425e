// gdn_probs.cu - from logits to probabilities over token trees (penalties for
// repeated tokens along each node's path, biases, grammar masks, temperature,
// softmax), and the commit of the accepted path's tokens to the history that the
// penalties read.
//
// Mathematics.  p_y = 2^(c (x_y - m)) f with m the largest x of a warp's tokens, c =
// log2(e) / T and f = 2^(c (m - M)) / sum over all of them: one exponential an element,
// taken against the warp's own maximum and kept, so that the row's warps exchange their
// (m, sum) only once, through distributed shared memory.  x is formed in the documented order with one rounding a step (the
// intrinsics keep products and sums apart), so that equal inputs give equal x and a
// tie is a tie.
//
// Mapping.  Few rows: a cluster of CTAs takes a row, each CTA runs of up to 16384 tokens
// whose x, then 2^(..), stay in registers (four groups of 8 a thread; of 64 registers, for two CTAs an SM, 32 bytes
// spill with 16-bit logits and 104 with fp32): the row is
// read once and written once, 6 bytes a token with 16-bit logits.  (A larger vocabulary
// than 16 slices hold reads the rest of each slice again for every pass.)  The logits are
// requested before the row's sequence is looked up.  Bound by latency: look-ups, loads, one
// exchange, stores; 16 rows of 131,072 tokens take 14 us, one 8 (fp32 logits 15; of 151,936 tokens, by clusters of 16,
// 19 and 21; of 248,320 23 and 26).  More rows than that: the second kernel, below.  Few tokens are touched by a path or a bias: a bitmap of groups of 8 in
// shared memory says which, and only those look into the lists; the history's 16 bits a token
// come from L2 for all of a sequence's nodes but the first.
#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "gdn_attn.h"
#include "gdn_tma.h"

namespace {
namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32, kGroups = 4, kMaxCluster = 16;
constexpr int kSlice = kThreads * kGroups * 8;  // tokens that a CTA keeps in registers
constexpr int kMarkBits = 2048;                 // the bitmap: a slice's groups, modulo (a larger slice's share bits)

struct ProbsArgs {
    const void *__restrict__ logits;
    int64_t l_stride;
    const int32_t *__restrict__ tokens, *__restrict__ parents, *__restrict__ node_off, *__restrict__ slot_map;
    const uint16_t *__restrict__ history;
    int64_t h_stride;
    const float *__restrict__ repetition, *__restrict__ frequency, *__restrict__ presence, *__restrict__ temperature;
    const int32_t *__restrict__ bias_off, *__restrict__ bias_token;
    const float *__restrict__ bias_value;
    const uint32_t *__restrict__ mask;
    int64_t mask_stride;
    const int32_t *__restrict__ mask_row;
    float *__restrict__ p;
    int64_t p_stride;
    int32_t *status;
    int S, N, P, V, max_nodes, n_bias, n_masks;
    int groups, per;  // groups of 8 tokens: of a row, of a CTA (a multiple of 32)
};

// What a row needs beside its logits.
struct Row {
    float r, inv_r, f, g, t;
    int slot, mask, b0, b1, n_path;  // slot, mask: -1 for none
    int err;
};

// A warp's (m, sum, place, NaN) as its cluster sees it.
struct __align__(16) Part {  // (sent in one piece)
    float m, sum;
    int best, nan;
};

template <typename T> struct Raw { uint4 v; };
template <> struct Raw<float> { uint4 v, w; };

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T *row, int g) {
    Raw<T> r;
    r.v = *reinterpret_cast<const uint4 *>(row + int64_t(g) * 8);
    if constexpr (std::is_same<T, float>::value) r.w = *reinterpret_cast<const uint4 *>(row + int64_t(g) * 8 + 4);
    return r;
}
template <typename T>
__device__ __forceinline__ void unpack_raw(const Raw<T> &r, float (&x)[8]) {
    if constexpr (std::is_same<T, float>::value) {
        const uint32_t w[8] = {r.v.x, r.v.y, r.v.z, r.v.w, r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e]);
    } else {
        gdn::unpack8<T>(r.v, x);
    }
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One token's penalties; h: its 16 bits of history.
__device__ __forceinline__ float penalised(float x, uint32_t h, const Row &row) {
    const uint32_t c = h & 0x7fffu;
    float y = __fmul_rn(x, x > 0.f ? row.inv_r : row.r);
    // (c as a float: it fits below 2^23)
    y = __fsub_rn(y, __fmul_rn(row.f, __uint_as_float(0x4b000000u | c) - 8388608.f));
    y = c ? __fsub_rn(y, row.g) : y;
    y = fabsf(x) <= FLT_MAX ? fminf(fmaxf(y, -FLT_MAX), FLT_MAX) : y;
    return h ? y : x;
}

// Where a CTA's groups of 8 tokens lie: runs of 256, dealt out over the cluster.  (What a part of the vocabulary costs -
// frequent tokens, which the history holds, are neighbours as a rule - all of them share.)
constexpr int kRun = 256;
struct Slice {
    int C, rank, groups;
    __device__ __forceinline__ int group(int local) const { return ((local / kRun) * C + rank) * kRun + local % kRun; }
    // the local index of a token's group; -1 for another CTA's
    __device__ __forceinline__ int local_of(int token) const {
        const int g = token >> 3, run = g / kRun;
        return run % C == rank ? run / C * kRun + g % kRun : -1;
    }
};

// What a row needs beside its logits; the path's tokens to `path` (a whole warp).
__device__ __forceinline__ Row read_row(const ProbsArgs &a, int n, int *path_out) {
    const unsigned full = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const int s = gdn::find_sequence(a.node_off, a.S, n);
    const int n0 = a.node_off[s], n1 = a.node_off[s + 1], i = n - n0;
    Row r{1.f, 1.f, 0.f, 0.f, 1.f, -1, -1, 0, 0, 0, 0};
    if (i < 0 || n >= n1 || n1 > a.N || n1 - n0 > a.max_nodes || n0 < 0 || (s == 0 && n0 != 0) || (s == a.S - 1 && n1 != a.N)) {
        r.err = GDN_DEV_BAD_NODE_OFF;
        return r;
    }
    if (a.temperature) r.t = a.temperature[s];
    if (a.mask) {
        r.mask = a.mask_row ? a.mask_row[n] : n;
        if (r.mask < -1 || r.mask >= a.n_masks) r.err = GDN_DEV_BAD_MASK;
    }
    if (a.bias_off) {
        r.b0 = a.bias_off[s];
        r.b1 = a.bias_off[s + 1];
        if (r.b0 < 0 || r.b1 < r.b0 || r.b1 > a.n_bias) {
            r.err = GDN_DEV_BAD_BIAS;
            r.b0 = r.b1 = 0;
        }
    }
    if (a.repetition || a.frequency || a.presence) {
        if (a.repetition) r.r = a.repetition[s];
        r.inv_r = __fdiv_rn(1.f, r.r);
        if (a.frequency) r.f = a.frequency[s];
        if (a.presence) r.g = a.presence[s];
        if (a.history) {
            r.slot = a.slot_map[s];
            if (r.slot < 0 || r.slot >= a.P) r.err = GDN_DEV_BAD_SLOT;
        }
        // the path: nodes 0 .. i of the sequence, two to a lane (i < 64)
        const int p_lo = lane <= i ? a.parents[n0 + lane] : -1, p_hi = lane + 32 <= i ? a.parents[n0 + lane + 32] : -1;
        const int t_lo = lane <= i ? a.tokens[n0 + lane] : 0, t_hi = lane + 32 <= i ? a.tokens[n0 + lane + 32] : 0;
        unsigned long long path = 0;
        for (int cur = i; cur >= 0;) {
            path |= 1ull << cur;
            const int p = __shfl_sync(full, cur < 32 ? p_lo : p_hi, cur & 31);
            if (p < -1 || p >= cur) {
                r.err = GDN_DEV_BAD_PARENT;
                break;
            }
            cur = p;
        }
        bool bad = false;
        for (int half = 0; half < 2; ++half) {
            const int x = lane + 32 * half, t = half ? t_hi : t_lo;
            if (!((path >> x) & 1)) continue;
            bad |= t < 0 || t >= a.V;
            path_out[__popcll(path & ((1ull << x) - 1))] = t;
        }
        if (__any_sync(full, bad)) r.err = GDN_DEV_BAD_TOKEN;
        r.n_path = __popcll(path);
    }
    return r;
}

// A row looks at its own sequence's offsets; the first CTA looks at all of them (threads t of n), those that no row comes to
// among them.
__device__ __forceinline__ void check_offsets(const ProbsArgs &a, int t, int n) {
    if (blockIdx.x != 0) return;
    const int err = gdn::check_node_off(a.node_off, a.S, a.N, a.max_nodes, t, n);
    if (err) gdn::record_status(a.status, err);
}

// touch(token) for the biases, thread t of n; whether its share of them is out of order.
template <typename Touch>
__device__ __forceinline__ bool for_biases(const ProbsArgs &a, const Row &row, int t, int n, Touch &&touch) {
    bool bad = false;
    for (int k = row.b0 + t; k < row.b1; k += n) {
        const int y = a.bias_token[k];
        if (y < 0 || y >= a.V || (k > row.b0 && a.bias_token[k - 1] >= y)) bad = true;
        else touch(y);
    }
    return bad;
}
// Marks the groups that the path and the biases touch, thread t of n; whether its share of the biases is out of order.
__device__ __forceinline__ bool mark_groups(const ProbsArgs &a, const Slice &sl, const Row &row, const int *path, uint32_t *mark, int t, int n) {
    auto touch = [&](int token) {
        const int local = sl.local_of(token);
        if (local >= 0) atomicOr(mark + ((local >> 5) & (kMarkBits / 32 - 1)), 1u << (local & 31));
    };
    for (int k = t; k < row.n_path; k += n) touch(path[k]);
    return for_biases(a, row, t, n, touch);
}

// x of group g; mark: the word with its bit.
template <typename T>
__device__ __forceinline__ void form(const ProbsArgs &a, const Row &row, const int *path, uint32_t mark, const Raw<T> &in, const uint4 &h,
                                     uint32_t allowed, int g, float (&x)[8]) {
    unpack_raw<T>(in, x);
    uint32_t hw[4] = {h.x, h.y, h.z, h.w};
    const bool marked = (mark >> (g & 31)) & 1;
    if (marked) {
        for (int k = 0; k < row.n_path; ++k) {
            const int t = path[k];
            if (t >> 3 != g) continue;
            const int sh = 16 * (t & 1);
#pragma unroll
            for (int z = 0; z < 4; ++z)  // (as a sum for all: a choice of one would put them in memory)
                hw[z] += z == ((t & 7) >> 1) && ((hw[z] >> sh) & 0x7fffu) != 0x7fffu ? 1u << sh : 0u;
        }
    }
    if (hw[0] | hw[1] | hw[2] | hw[3]) {
        // (few tokens have a history, so a warp skips most of the eight)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t he = (hw[e >> 1] >> (16 * (e & 1))) & 0xffffu;
            if (__builtin_expect(he != 0, 0)) x[e] = penalised(x[e], he, row);
        }
    }
    if (marked && row.b1 > row.b0) {
        int lo = row.b0, hi = row.b1;  // the first entry of the group or after it
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.bias_token[mid] < 8 * g) lo = mid + 1;
            else hi = mid;
        }
        for (; lo < row.b1; ++lo) {
            const int t = a.bias_token[lo];
            if (t >> 3 != g) break;
            const float b = a.bias_value[lo];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __fadd_rn(x[e], e == (t & 7) ? b : 0.f);
        }
    }
    const int left = a.V - 8 * g;  // tokens of the group
    if (left < 8) allowed &= (1u << left) - 1u;
    if (allowed != 0xffu) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (!((allowed >> e) & 1)) x[e] = -INFINITY;
    }
}

// (c is neither 0 nor infinite, so that x = -inf gives 0)
__device__ __forceinline__ float scale_of(const Row &row) { return fminf(fmaxf(__fdiv_rn(1.4426950408889634f, row.t), FLT_MIN), FLT_MAX); }
__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
// m: the warp's maximum (with -inf taken as 0, so that nothing is subtracted from it; NaN stays NaN)
__device__ __forceinline__ float weight(float x, float m, float c) { return exp2_fast(__fmul_rn(__fsub_rn(x, m == -INFINITY ? 0.f : m), c)); }

template <int n>
__device__ __forceinline__ void look(const float (&y)[n], float m, int first, Part &mine) {
#pragma unroll
    for (int e = n - 1; e >= 0; --e) {
        if (y[e] == m && m > -INFINITY) mine.best = min(mine.best, first + e);
        mine.nan |= y[e] != y[e];
    }
}

// The row's, from every warp of the cluster in a fixed order.
struct Whole {
    float f;  // 1 / sum, 0 where nothing is left
    int best, nan;
    float m;
};
__device__ __forceinline__ Whole whole_of(const Part *parts, int n, float c) {
    const int lane = threadIdx.x & 31;
    Part all{-INFINITY, 0.f, INT32_MAX, 0};
    for (int k = lane; k < n; k += 32) all.m = fmaxf(all.m, parts[k].m);
    const float M = warp_max(all.m);
    for (int k = lane; k < n; k += 32) {
        const Part q = parts[k];
        if (q.m == M) all.best = min(all.best, q.best);
        all.nan |= q.nan;
        all.sum += q.m == -INFINITY ? q.sum : q.sum * exp2_fast(__fmul_rn(__fsub_rn(q.m, M), c));
    }
    const float total = gdn::warp_sum(all.sum);
    return {total == 0.f ? 0.f : __fdividef(1.f, total), __reduce_min_sync(0xffffffffu, all.best),
            int(__reduce_or_sync(0xffffffffu, unsigned(all.nan))), M};
}

__device__ __forceinline__ void store8(const ProbsArgs &a, float *prow, int g, const float (&y)[8]) {
    const int left = a.V - 8 * g;
    float *to = prow + int64_t(g) * 8;
    if (left >= 8) {
        *reinterpret_cast<float4 *>(to) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4 *>(to + 4) = make_float4(y[4], y[5], y[6], y[7]);
    } else {
#pragma unroll
        for (int z = 0; z < 8; ++z)
            if (z < left) to[z] = y[z];
    }
}
__device__ __forceinline__ void store_one_hot(const ProbsArgs &a, const Slice &sl, float *prow, const Whole &w) {
    const float no = w.nan ? __uint_as_float(0x7fffffffu) : 0.f, yes = w.nan ? no : 1.f;
#pragma unroll 1
    for (int local = threadIdx.x; local < a.per; local += kThreads) {
        const int g = sl.group(local);
        if (g >= sl.groups) break;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = 8 * g + e == w.best ? yes : no;
        store8(a, prow, g, y);
    }
}

// A cluster to a row: as many as the GPU holds at once at most, or (kRest) of a vocabulary that the cluster's registers do not hold.
template <typename T, bool kRest>
__global__ void __launch_bounds__(kThreads, 2) logits_probs_kernel(const ProbsArgs a) {
    __shared__ Row row_s;
    __shared__ int path_s[gdn::kMaxSeqNodes];
    __shared__ uint32_t mark[kMarkBits / 32];
    __shared__ Part parts[kMaxCluster * kWarps];
    cg::cluster_group cl = cg::this_cluster();
    gdn::grid_dep_launch();
    const Slice sl{int(cl.num_blocks()), int(cl.block_rank()), a.groups};
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = int(blockIdx.x) / sl.C;
    auto arrived = cl.barrier_arrive();  // every CTA of the cluster runs before one writes to another
    gdn::grid_dep_wait();

    const T *lrow = static_cast<const T *>(a.logits) + int64_t(n) * a.l_stride;
    auto there = [&](int local) { return local < a.per && sl.group(local) < sl.groups; };
    Raw<T> raw[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
        if (there(k * kThreads + tid)) raw[k] = load_raw<T>(lrow, sl.group(k * kThreads + tid));
    if (tid < kMarkBits / 32) mark[tid] = 0;
    if (warp == 0) {
        const Row r = read_row(a, n, path_s);
        if (lane == 0) row_s = r;
    } else {
        check_offsets(a, tid - 32, kThreads - 32);
    }
    __syncthreads();
    const Row row = row_s;
    const uint16_t *hrow = row.slot >= 0 ? a.history + int64_t(row.slot) * a.h_stride : nullptr;
    const unsigned char *mrow =
        row.mask >= 0 ? reinterpret_cast<const unsigned char *>(a.mask + int64_t(row.mask) * a.mask_stride) : nullptr;
    auto history_of = [&](int g) { return hrow ? *reinterpret_cast<const uint4 *>(hrow + int64_t(g) * 8) : make_uint4(0, 0, 0, 0); };
    auto allowed_of = [&](int g) { return mrow ? uint32_t(mrow[g]) : 0xffu; };
    uint4 h[kGroups];
    uint32_t allowed[kGroups];
    if (!row.err) {
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
            if (there(k * kThreads + tid)) {
                h[k] = history_of(sl.group(k * kThreads + tid));
                allowed[k] = allowed_of(sl.group(k * kThreads + tid));
            }
    }
    const bool bad = !row.err && mark_groups(a, sl, row, path_s, mark, tid, kThreads);
    const int err = row.err ? row.err : __syncthreads_or(bad) ? GDN_DEV_BAD_TOKEN : 0;  // (row.err is the same for all threads)
    if (err) {
        if (tid == 0 && sl.rank == 0) gdn::record_status(a.status, err);
        cl.barrier_wait(std::move(arrived));
        return;  // the cluster's other CTAs have read the same and leave too
    }

    auto mark_of = [&](int local) { return mark[(local >> 5) & (kMarkBits / 32 - 1)]; };
    // the groups that registers do not hold
    auto for_rest = [&](auto &&body) {
        if constexpr (kRest) {
#pragma unroll 1
            for (int local = kGroups * kThreads + tid; there(local); local += kThreads) {
                const int g = sl.group(local);
                float x[8];
                form<T>(a, row, path_s, mark_of(local), load_raw<T>(lrow, g), history_of(g), allowed_of(g), g, x);
                body(g, x);
            }
        }
    };
    float x[kGroups][8];
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const int local = k * kThreads + tid;
        if (there(local)) {
            form<T>(a, row, path_s, mark_of(local), raw[k], h[k], allowed[k], sl.group(local), x[k]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, x[k][e]);
    }
    for_rest([&](int, float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, y[e]);
    });
    m = warp_max(m);
    const bool greedy = !(row.t > 0.f);
    const float c = scale_of(row);
    Part mine{m, 0.f, INT32_MAX, 0};
    if (greedy) {
#pragma unroll
        for (int k = 0; k < kGroups; ++k) look(x[k], m, 8 * sl.group(k * kThreads + tid), mine);
        for_rest([&](int g, float (&y)[8]) { look(y, m, 8 * g, mine); });
        mine.best = __reduce_min_sync(0xffffffffu, mine.best);
        mine.nan = __reduce_or_sync(0xffffffffu, mine.nan);
    } else {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[k][e] = weight(x[k][e], m, c);
                s += x[k][e];
            }
        for_rest([&](int, float (&y)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s += weight(y[e], m, c);
        });
        mine.sum = gdn::warp_sum(s);
    }
    cl.barrier_wait(std::move(arrived));
    if (lane < sl.C) *cl.map_shared_rank(parts + sl.rank * kWarps + warp, lane) = mine;
    cl.sync();
    const Whole w = whole_of(parts, sl.C * kWarps, c);
    // (a NaN total stays)
    const float f = m == -INFINITY ? w.f * 0.f : exp2_fast(__fmul_rn(__fsub_rn(m, w.m), c)) * w.f;
    float *prow = a.p + int64_t(n) * a.p_stride;
    if (greedy) {
        store_one_hot(a, sl, prow, w);
        return;
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const int local = k * kThreads + tid;
        if (there(local)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] *= f;
            store8(a, prow, sl.group(local), x[k]);
        }
    }
    for_rest([&](int g, float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = weight(y[e], m, c) * f;
        store8(a, prow, g, y);
    });
}

// ---- more rows than the GPU holds at once --------------------------------------------------
//
// With a row in a cluster's registers a CTA's life is a chain of ~25,000 cycles (look-ups, loads, an exchange between
// eight CTAs that are never equally far, stores), of which its memory's share of the GPU is 4,600, and registers hold two
// CTAs an SM: 1024 rows of 131,072 took 445 us, and 385 with the next rows' logits copied ahead.  Here a CTA of an SM of
// its own keeps 128 KB of logits (two CTAs a row of 131,072 bf16) in shared memory and goes over them twice: maxima and
// sums, an exchange, and the probabilities, forming x again.  A chunk of the next row is copied as soon as a chunk of
// this one has been read for the last time, so loads and stores share the time; the next row is looked up by a warp that
// waits for the exchange.  1024 rows of 131,072 with penalties, biases and masks take 338-384 us so, without any of them
// 228-238, against 124 of memory: bound by instructions (~190 for 8 tokens a lane and pass without them), since x is formed
// twice; DRAM is at a third.  Beyond 131,072 bf16 (65,536 fp32) tokens a row is four CTAs or more, which work in step:
// 151,936 take 479 us (floor 144), 248,320 643 (235); fp32 logits of 131,072 430-451 (164), of 151,936, by eight CTAs with
// two or three of their four chunks in use, 830 (190), of 248,320, by eight too, 972 (311).
struct Head {
    Row row;
    int path[gdn::kMaxSeqNodes];
    uint32_t mark[256];  // a bit for each of the CTA's groups
};
constexpr int kRowThreads = 1024, kRowWarps = kRowThreads / 32;
template <typename T>
struct RowChunks {
    static constexpr uint32_t kBytes = kRowThreads * 8 * sizeof(T);  // a chunk: a group a thread
    static constexpr int kChunks = int(131072 / kBytes), kTokens = kChunks * kRowThreads * 8;
};

__device__ __forceinline__ bool wait_rows(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    bool ok = gdn::mbar_try_wait(bar, parity);
    if (!ok && !*abort_flag) ok = gdn::mbar_wait_bounded(bar, parity);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *abort_flag = 1;
    return ok;
}
// `v` to the same place of CTA `rank`'s shared memory, counted by the same barrier there
__device__ __forceinline__ void send(const Part *to, uint64_t *bar, int rank, const Part &v) {
    uint32_t ra, rb;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(gdn::smem_addr(to)), "r"(rank));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rb) : "r"(gdn::smem_addr(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(ra),
                 "r"(__float_as_uint(v.m)), "r"(__float_as_uint(v.sum)), "r"(v.best), "r"(v.nan), "r"(rb)
                 : "memory");
}

// Counts a warp that has read a chunk for the last time (one lane, the warp together before it); whether it is the last of
// them.  With release and acquire, so that all warps' reads come before what the last one does next: the copy over the chunk
// and the arrival at its barrier, by which they also come before what is done after a wait for that copy (look_up over the
// head of the row before).  An mbarrier that says who came last takes 1024 rows without penalties from 238 to 246 us.
__device__ __forceinline__ bool last_reader(int *count) {
    int before;
    asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(before) : "r"(gdn::smem_addr(count)) : "memory");
    return before == kRowWarps - 1;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads, 1) logits_probs_rows_kernel(const ProbsArgs a) {
    using K = RowChunks<T>;
    extern __shared__ __align__(128) unsigned char chunks[];
    __shared__ Head heads[2];
    __shared__ uint64_t head_bar[2], full_bar[K::kChunks], part_bar[2];
    __shared__ Part parts[2][kMaxCluster * kRowWarps];
    __shared__ int read_s[K::kChunks];  // warps that have read a chunk for the last time
    __shared__ int abort_s;
    volatile int *abort_flag = &abort_s;
    const unsigned full = 0xffffffffu;
    cg::cluster_group cl = cg::this_cluster();
    gdn::grid_dep_launch();
    const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int clusters = int(gridDim.x) / C, mine_c = int(blockIdx.x) / C;
    const int first = int(int64_t(a.N) * mine_c / clusters), last = int(int64_t(a.N) * (mine_c + 1) / clusters);
    // chunk k of the row is the CTA's (k / C)th
    const int total_chunks = (a.groups + kRowThreads - 1) / kRowThreads, mine_n = (total_chunks - rank + C - 1) / C;
    if (tid == 0) {
        for (int i = 0; i < K::kChunks; ++i) {
            gdn::mbar_init(full_bar + i, 1);
            read_s[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            gdn::mbar_init(head_bar + i, 1);
            gdn::mbar_init(part_bar + i, 1);
        }
        gdn::fence_mbar_init();
        abort_s = 0;
    }
    cl.sync();  // every CTA's barriers are there before one of another sends to them
    gdn::grid_dep_wait();
    check_offsets(a, tid, kRowThreads);

    auto load = [&](int n, int k) {  // one thread
        const int g = (k * C + rank) * kRowThreads;
        const uint32_t bytes = uint32_t(min(kRowThreads, a.groups - g)) * 8 * sizeof(T);
        gdn::mbar_arrive_expect_tx(full_bar + k, bytes);
        gdn::bulk_load(chunks + k * K::kBytes, static_cast<const T *>(a.logits) + int64_t(n) * a.l_stride + int64_t(g) * 8, bytes, full_bar + k);
    };
    auto look_up = [&](int n) {  // a warp
        Head &hd = heads[n & 1];
#pragma unroll
        for (int i = 0; i < 8; ++i) hd.mark[32 * i + lane] = 0;
        Row r = read_row(a, n, hd.path);
        __syncwarp();
        bool bad = false;
        if (!r.err) {
            auto touch = [&](int token) {
                const int g = token >> 3, k = g / kRowThreads;
                if (k % C == rank) atomicOr(hd.mark + ((k / C * kRowThreads + g % kRowThreads) >> 5), 1u << (g & 31));
            };
            for (int k = lane; k < r.n_path; k += 32) touch(hd.path[k]);
            bad = for_biases(a, r, lane, 32, touch);
        }
        if (__any_sync(full, bad)) r.err = GDN_DEV_BAD_TOKEN;
        if (lane == 0) {
            hd.row = r;
            if (r.err && rank == 0) gdn::record_status(a.status, r.err);
        }
        __syncwarp();
        if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(gdn::smem_addr(head_bar + (n & 1))) : "memory");
    };
    if (first < last) {
        if (warp == 0) {
            if (lane == 0) {
                asm volatile("fence.proxy.async;" ::: "memory");  // what earlier kernels wrote, for the copies
                for (int k = 0; k < mine_n; ++k) load(first, k);
            }
            __syncwarp();
            look_up(first);
        }
    }
    int sent = 0;  // rows whose parts have been exchanged
    bool ok = true;
    for (int n = first; n < last; ++n) {
        ok = wait_rows(head_bar + (n & 1), uint32_t((n - first) >> 1) & 1, abort_flag);
        if (!ok) break;
        const Head &hd = heads[n & 1];
        const Row row = hd.row;
        const uint32_t phase = uint32_t(n - first) & 1;
        const uint16_t *hrow = row.slot >= 0 ? a.history + int64_t(row.slot) * a.h_stride : nullptr;
        const unsigned char *mrow =
            row.mask >= 0 ? reinterpret_cast<const unsigned char *>(a.mask + int64_t(row.mask) * a.mask_stride) : nullptr;
        auto group = [&](int k) { return (k * C + rank) * kRowThreads + tid; };
        auto x_of = [&](int k, int g, float (&x)[8]) {
            const uint4 h = hrow ? *reinterpret_cast<const uint4 *>(hrow + int64_t(g) * 8) : make_uint4(0, 0, 0, 0);
            form<T>(a, row, hd.path, hd.mark[k * (kRowThreads / 32) + warp], load_raw<T>(reinterpret_cast<const T *>(chunks + k * K::kBytes), tid), h,
                    mrow ? mrow[g] : 0xffu, g, x);
        };
        const bool greedy = !(row.t > 0.f);
        const float c = scale_of(row);
        Whole w{0.f, 0, 0, 0.f};
        if (row.err) {
            // (no work, but the waits: a chunk that has come in says that all warps are done with the row before)
            for (int k = 0; k < mine_n && ok; ++k) ok = wait_rows(full_bar + k, phase, abort_flag);
            if (!ok) break;
        } else {
            // ---- maxima and sums, a thread's own as they come ----------------------------------
            Part mine{-INFINITY, 0.f, INT32_MAX, 0};
#pragma unroll 1
            for (int k = 0; k < mine_n; ++k) {
                ok = wait_rows(full_bar + k, phase, abort_flag);
                if (!ok) break;
                const int g = group(k);
                if (g >= a.groups) continue;
                float x[8];
                x_of(k, g, x);
                float m = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
                if (greedy) {
                    if (m > mine.m) {
                        mine.m = m;
                        mine.best = INT32_MAX;
                    }
                    look(x, mine.m, 8 * g, mine);
                } else {
                    m = fmaxf(m, mine.m);
                    float s = mine.sum * weight(mine.m, m, c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s += weight(x[e], m, c);
                    mine.m = m;
                    mine.sum = s;
                }
            }
            if (!ok) break;
            const float m = warp_max(mine.m);
            if (greedy) {
                mine.best = __reduce_min_sync(full, mine.m == m ? mine.best : INT32_MAX);
                mine.nan = __reduce_or_sync(full, mine.nan);
            } else {
                mine.sum = gdn::warp_sum(mine.sum * weight(mine.m, m, c));
            }
            mine.m = m;
            // Two places in turn: a warp sends a row's part when it has read those of the row before, so what comes in for
            // a row finds the place of two rows before read by all.
            const int z = sent & 1;
            if (tid == 0) gdn::mbar_arrive_expect_tx(part_bar + z, uint32_t(C * kRowWarps * sizeof(Part)));
            if (lane < C) send(parts[z] + rank * kRowWarps + warp, part_bar + z, lane, mine);
            __syncwarp();
        }
        // (its place is that of the row before, which no warp reads any more: every chunk of this row has come in)
        if (n + 1 < last && warp == (n & (kRowWarps - 1))) look_up(n + 1);
        if (!row.err) {
            const int z = sent & 1;
            ok = wait_rows(part_bar + z, uint32_t(sent >> 1) & 1, abort_flag);
            if (!ok) break;
            ++sent;
            w = whole_of(parts[z], C * kRowWarps, c);
        }
        // ---- the probabilities; a chunk that all warps have read makes room for the next row's ----
        float *prow = a.p + int64_t(n) * a.p_stride;
        const float no = w.nan ? __uint_as_float(0x7fffffffu) : 0.f, yes = w.nan ? no : 1.f;
#pragma unroll 1
        for (int k = 0; k < mine_n; ++k) {
            const int g = group(k);
            const bool there = g < a.groups && !row.err;
            float x[8];
            if (there && !greedy) x_of(k, g, x);
            __syncwarp();
            if (lane == 0 && n + 1 < last && last_reader(read_s + k)) {
                read_s[k] = 0;
                load(n + 1, k);
            }
            if (there) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = greedy ? (8 * g + e == w.best ? yes : no) : weight(x[e], w.m, c) * w.f;
                store8(a, prow, g, x);
            }
        }
    }
    __syncwarp();
    __syncthreads();
    // (a row that was not come to after a wait ran out: its copies end before the CTA does)
    if (abort_s && tid < mine_n) {
        gdn::mbar_wait_bounded(full_bar + tid, 0, 1000000);
        gdn::mbar_wait_bounded(full_bar + tid, 1, 1000000);
    }
    if (tid == 0 && abort_s) gdn::record_status(a.status, GDN_DEV_TIMEOUT);
    cl.sync();  // nothing is on its way into a CTA that has left
}

// ---- the history's commit ------------------------------------------------------------------

struct TokenArgs {
    const int32_t *__restrict__ tokens, *__restrict__ accepted, *__restrict__ parents, *__restrict__ node_off, *__restrict__ slot_map;
    uint16_t *history;
    int64_t h_stride;
    int32_t *status;
    int S, N, P, V, max_nodes, prompt;
};

// Whether sequence s commits anything.
__device__ __forceinline__ bool commits(const TokenArgs &a, int s) {
    return a.accepted ? a.accepted[s] >= 0 : a.node_off[s + 1] > a.node_off[s];
}

// The path root .. acc as a mask of nodes (a whole warp); *err set for a parent that is not before its child.
__device__ __forceinline__ unsigned long long token_path(const TokenArgs &a, int n0, int acc, int *err) {
    const int lane = threadIdx.x & 31;
    const int p_lo = lane <= acc ? a.parents[n0 + lane] : -1, p_hi = lane + 32 <= acc ? a.parents[n0 + lane + 32] : -1;
    unsigned long long path = 0;
    for (int cur = acc; cur >= 0;) {
        path |= 1ull << cur;
        const int p = __shfl_sync(0xffffffffu, cur < 32 ? p_lo : p_hi, cur & 31);
        if (p < -1 || p >= cur) {
            *err = GDN_DEV_BAD_PARENT;
            break;
        }
        cur = p;
    }
    return path;
}

// CTAs of a sequence (y), as in the commit itself: one for a round's few nodes, more for a prompt's many tokens.
__global__ void __launch_bounds__(256) token_preflight_kernel(const TokenArgs a) {
    __shared__ unsigned long long path_s;
    __shared__ int err_s;
    gdn::grid_dep_launch();
    gdn::grid_dep_wait();
    const int s = blockIdx.x, tid = threadIdx.x;
    const int n0 = a.node_off[s], n1 = a.node_off[s + 1], ns = n1 - n0;
    if (tid < 32) {
        int err = 0;
        unsigned long long path = ~0ull;
        if (n0 < 0 || n1 < n0 || n1 > a.N || (s == 0 && n0 != 0) || (s == a.S - 1 && n1 != a.N) || (a.accepted && ns > a.max_nodes)) {
            err = GDN_DEV_BAD_NODE_OFF;
        } else if (a.accepted) {
            const int acc = a.accepted[s];
            if (acc < -1 || acc >= ns) err = GDN_DEV_BAD_ACCEPTED;
            else path = token_path(a, n0, acc, &err);
        }
        if (tid == 0) {
            path_s = path;
            err_s = err;
        }
    }
    __syncthreads();
    int err = err_s;  // the same for all threads
    if (!err && commits(a, s)) {
        const int slot = a.slot_map[s];
        if (slot < 0 || slot >= a.P) {
            err = GDN_DEV_BAD_SLOT;
        } else {
            bool bad = false, dup = false;
            for (int k = 256 * blockIdx.y + tid; k < ns; k += 256 * gridDim.y) {
                const int t = a.tokens[n0 + k];
                bad |= (!a.accepted || ((path_s >> k) & 1)) && (t < 0 || t >= a.V);
            }
            for (int s2 = tid; s2 < a.S && blockIdx.y == 0; s2 += 256) dup |= s2 != s && a.slot_map[s2] == slot && commits(a, s2);
            if (__syncthreads_or(bad)) err = GDN_DEV_BAD_TOKEN;
            else if (__syncthreads_or(dup)) err = GDN_DEV_DUP_SLOT;
        }
    }
    if (err && tid == 0) gdn::record_status(a.status, err);
}

__global__ void __launch_bounds__(256) token_commit_kernel(const TokenArgs a) {
    __shared__ unsigned long long path_s;
    gdn::grid_dep_launch();
    gdn::grid_dep_wait();
    if (*reinterpret_cast<volatile int32_t *>(a.status) != 0) return;
    const int s = blockIdx.x, tid = threadIdx.x;
    if (!commits(a, s)) return;
    const int n0 = a.node_off[s], ns = a.node_off[s + 1] - n0;
    if (a.accepted) {
        if (tid < 32) {
            int err = 0;
            const unsigned long long path = token_path(a, n0, a.accepted[s], &err);
            if (tid == 0) path_s = path;
        }
        __syncthreads();
    }
    uint16_t *row = a.history + int64_t(a.slot_map[s]) * a.h_stride;
    for (int k = 256 * blockIdx.y + tid; k < ns; k += 256 * gridDim.y) {
        if (a.accepted && !((path_s >> k) & 1)) continue;
        const int t = a.tokens[n0 + k];
        unsigned int *w = reinterpret_cast<unsigned int *>(row + (t & ~1));
        const int sh = 16 * (t & 1);
        if (a.prompt) {
            atomicOr(w, 0x8000u << sh);
        } else {
            // (whole numbers: the order of a token's counts does not change their sum)
            unsigned int old = *reinterpret_cast<volatile unsigned int *>(w);
            while (((old >> sh) & 0x7fffu) != 0x7fffu) {
                const unsigned int seen = atomicCAS(w, old, old + (1u << sh));
                if (seen == old) break;
                old = seen;
            }
        }
    }
}

template <typename T>
int launch_probs(const ProbsArgs &args, int64_t rows, int vocab, cudaStream_t st) {
    ProbsArgs a = args;
    // A cluster whose registers hold the row, of more CTAs while there are few rows to fill the GPU with.  (Not all clusters of 16
    // find their places at once: one row of 131,072 takes 8.2 us with 16 CTAs and 9.9 with 8, 12 rows 10.9 and 12.3, 16 rows
    // 18.0 and 14.3.)
    const int sms = gdn::sm_count_current();
    if (sms < 1) return GDN_ERR_LAUNCH;
    int C = 1;
    while (C < kMaxCluster && (int64_t(C) * kSlice < vocab || (rows * 2 * C <= 2 * sms && vocab / (2 * C) >= 2048 && (C < 8 || rows <= 12)))) C *= 2;
    a.groups = int((int64_t(vocab) + 7) / 8);
    const bool rest = int64_t(C) * kSlice < vocab;
    auto k = rest ? logits_probs_kernel<T, true> : logits_probs_kernel<T, false>;
    cudaLaunchConfig_t cfg = {};
    // Rows that would come in several waves: CTAs that stay.  (Below 16384 tokens a row is less than a thread's share each.)
    const bool many = rows * C > 2 * sms && vocab >= 16384 && int64_t(vocab) <= int64_t(kMaxCluster) * RowChunks<T>::kTokens;
    if (many) {
        k = logits_probs_rows_kernel<T>;
        for (C = 1; int64_t(C) * RowChunks<T>::kTokens < vocab;) C *= 2;
        cfg.dynamicSmemBytes = 131072;
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(cfg.dynamicSmemBytes)) != cudaSuccess) return GDN_ERR_LAUNCH;
    }
    a.per = ((a.groups + kRun - 1) / kRun + C - 1) / C * kRun;
    if (C > 8 && cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return GDN_ERR_LAUNCH;
    if (rows * C > INT32_MAX) return GDN_ERR_DIMS;
    cfg.blockDim = dim3(many ? kRowThreads : kThreads);
    cfg.gridDim = dim3(unsigned(many ? C : rows * C));
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(C);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (many) {
        int clusters = 0;  // resident at once
        if (cudaOccupancyMaxActiveClusters(&clusters, k, &cfg) != cudaSuccess || clusters < 1) return GDN_ERR_LAUNCH;
        cfg.gridDim.x = unsigned(std::min<int64_t>(clusters, rows)) * unsigned(C);
    }
    return cudaLaunchKernelEx(&cfg, k, a) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace

extern "C" int gdn_logits_probs(const gdn_dims *dims, int vocab, int dtype, const void *logits, int64_t logits_stride,
                                const int32_t *tokens, const int32_t *parents, const int32_t *node_off,
                                const int32_t *slot_map, const uint16_t *history, int64_t history_stride,
                                const float *repetition, const float *frequency, const float *presence,
                                const float *temperature, const int32_t *bias_off, const int32_t *bias_token,
                                const float *bias_value, int n_bias, const uint32_t *mask, int64_t mask_stride,
                                const int32_t *mask_row, int n_masks, float *p, int64_t p_stride, int32_t *status,
                                void *stream) {
    int rc = gdn::check_dims(dims);
    if (rc) return rc;
    if (!status) return GDN_ERR_NULL;
    if (vocab < 1 || vocab > (1 << 28) || (dtype != GDN_BF16 && dtype != GDN_FP16 && dtype != GDN_FP32) || n_bias < 0 || n_masks < 0)
        return GDN_ERR_ARG;
    const int64_t S = dims->n_seqs, N = dims->n_nodes, P = dims->n_slots;
    if (S == 0 || N == 0) return GDN_OK;
    const bool counts = repetition || frequency || presence;
    if (!logits || !node_off || !p || (counts && (!tokens || !parents || (history && !slot_map)))) return GDN_ERR_NULL;
    if ((bias_off || bias_token || bias_value) && (!bias_off || (n_bias > 0 && (!bias_token || !bias_value)))) return GDN_ERR_NULL;
    const int64_t row8 = (int64_t(vocab) + 7) / 8 * 8, row4 = (int64_t(vocab) + 3) / 4 * 4, words = (int64_t(vocab) + 31) / 32;
    const int64_t most = int64_t(1) << 38;
    if (logits_stride < row8 || logits_stride % 8 || logits_stride > most || p_stride < row4 || p_stride % 4 || p_stride > most)
        return GDN_ERR_STRIDE;
    if (history && (history_stride < row8 || history_stride % 8 || history_stride > most)) return GDN_ERR_STRIDE;
    if (mask && (mask_stride < words || mask_stride > most)) return GDN_ERR_STRIDE;
    if (!gdn::aligned16(logits) || !gdn::aligned16(p) || !gdn::aligned16(history)) return GDN_ERR_ALIGN;
    const int64_t size = dtype == GDN_FP32 ? 4 : 2;
    const gdn::Span outs[] = {{p, gdn::strided_bytes(N, p_stride, row4)}};
    const gdn::Span ins[] = {{logits, size_t(((N - 1) * logits_stride + row8) * size)},
                             {tokens, size_t(N * 4)},
                             {parents, size_t(N * 4)},
                             {node_off, size_t((S + 1) * 4)},
                             {slot_map, size_t(S * 4)},
                             {history, history ? size_t(((P - 1) * history_stride + row8) * 2) : 0},
                             {repetition, size_t(S * 4)},
                             {frequency, size_t(S * 4)},
                             {presence, size_t(S * 4)},
                             {temperature, size_t(S * 4)},
                             {bias_off, size_t((S + 1) * 4)},
                             {bias_token, size_t(n_bias) * 4},
                             {bias_value, size_t(n_bias) * 4},
                             {mask, mask && n_masks > 0 ? size_t(((n_masks - 1) * mask_stride + words) * 4) : 0},
                             {mask_row, size_t(N * 4)},
                             {status, 4}};
    if ((rc = gdn::check_alias(outs, 1, ins, 16))) return rc;
    ProbsArgs a{logits, logits_stride, tokens, parents, node_off, slot_map, history, history_stride, repetition, frequency,
                presence, temperature, bias_off, bias_token, bias_value, mask, mask_stride, mask_row, p, p_stride, status,
                int(S), int(N), int(P), vocab, dims->max_seq_nodes, n_bias, n_masks, 0, 0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case GDN_BF16: return launch_probs<__nv_bfloat16>(a, N, vocab, st);
        case GDN_FP16: return launch_probs<__half>(a, N, vocab, st);
        default: return launch_probs<float>(a, N, vocab, st);
    }
}

extern "C" int gdn_token_commit(const gdn_dims *dims, int vocab, const int32_t *tokens, const int32_t *accepted,
                                const int32_t *parents, const int32_t *node_off, const int32_t *slot_map, int prompt,
                                uint16_t *history, int64_t history_stride, int32_t *status, void *stream) {
    int rc = gdn::check_dims(dims);
    if (rc) return rc;
    if (!status) return GDN_ERR_NULL;
    if (vocab < 1 || vocab > (1 << 28) || (prompt != 0 && prompt != 1)) return GDN_ERR_ARG;
    const int64_t S = dims->n_seqs, N = dims->n_nodes, P = dims->n_slots;
    if (S == 0 || N == 0) return GDN_OK;
    if (!tokens || !node_off || !slot_map || !history || (accepted && !parents)) return GDN_ERR_NULL;
    const int64_t row8 = (int64_t(vocab) + 7) / 8 * 8;
    if (history_stride < row8 || history_stride % 8 || history_stride > (int64_t(1) << 38)) return GDN_ERR_STRIDE;
    if (!gdn::aligned16(history)) return GDN_ERR_ALIGN;
    const gdn::Span outs[] = {{history, size_t(((P - 1) * history_stride + row8) * 2)}};
    const gdn::Span ins[] = {{tokens, size_t(N * 4)},          {accepted, size_t(S * 4)}, {parents, size_t(N * 4)},
                             {node_off, size_t((S + 1) * 4)}, {slot_map, size_t(S * 4)}, {status, 4}};
    if ((rc = gdn::check_alias(outs, 1, ins, 6))) return rc;
    TokenArgs a{tokens, accepted, parents, node_off, slot_map, history, history_stride, status, int(S), int(N), int(P), vocab,
                dims->max_seq_nodes, prompt};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(unsigned(S), unsigned(std::min<int64_t>((N + S * 256 - 1) / (S * 256), 64)));
    if (gdn::launch_pdl(token_preflight_kernel, grid, dim3(256), 0, st, a) != cudaSuccess) return GDN_ERR_LAUNCH;
    return gdn::launch_pdl(token_commit_kernel, grid, dim3(256), 0, st, a) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
