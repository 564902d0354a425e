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
// Mapping.  A cluster of CTAs takes a row, each CTA a slice of up to 16384 tokens
// whose x, then 2^(..), stay in registers (four groups of 8 a thread): the row is
// read once and written once, 6 bytes a token with 16-bit logits.  (A larger vocabulary
// than 16 slices hold reads the rest of each slice again for every pass.)  The logits are
// requested before the row's sequence is looked up.  Few tokens are touched by a path or
// a bias: a bitmap of groups of 8 in shared memory says which, and only those look into
// the lists; the history's 16 bits a token come from L2 for all of a sequence's nodes but
// the first.
#include <cooperative_groups.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "gdn_attn.h"

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
struct Part {
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

// kRest: the vocabulary is larger than the cluster's registers.
template <typename T, bool kRest>
__global__ void __launch_bounds__(kThreads, 2) logits_probs_kernel(const ProbsArgs a) {
    __shared__ Row row_s;
    __shared__ int path_s[gdn::kMaxSeqNodes];
    __shared__ uint32_t mark[kMarkBits / 32];
    __shared__ Part parts[kMaxCluster * kWarps];
    const unsigned full = 0xffffffffu;
    cg::cluster_group cl = cg::this_cluster();
    gdn::grid_dep_launch();
    const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = int(blockIdx.x) / C;
    // The row's groups in runs of 32, one a warp, dealt out over the cluster's warps: what a part of the vocabulary costs
    // (frequent tokens, which the history holds, are neighbours as a rule) all of them share.
    auto group = [&](int local) { return ((local >> 5) * C + rank) * 32 + (local & 31); };
    const int locals = a.per;
    auto arrived = cl.barrier_arrive();  // every CTA of the cluster runs before one writes to another
    gdn::grid_dep_wait();

    const T *lrow = static_cast<const T *>(a.logits) + int64_t(n) * a.l_stride;
    Raw<T> raw[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const int g = group(k * kThreads + tid);
        if (k * kThreads + tid < locals && g < a.groups) raw[k] = load_raw<T>(lrow, g);
    }

    // ---- the row's sequence, its path and its lists ---------------------------------
    const bool counts = a.repetition || a.frequency || a.presence;
    if (tid < kMarkBits / 32) mark[tid] = 0;
    if (warp == 0) {
        const int s = gdn::find_sequence(a.node_off, a.S, n);
        const int n0 = a.node_off[s], n1 = a.node_off[s + 1], i = n - n0;
        Row r{1.f, 1.f, 0.f, 0.f, 1.f, -1, -1, 0, 0, 0, 0};
        if (i < 0 || n >= n1 || n1 > a.N || n1 - n0 > a.max_nodes || n0 < 0 || (s == 0 && n0 != 0) || (s == a.S - 1 && n1 != a.N)) {
            r.err = GDN_DEV_BAD_NODE_OFF;
        } else {
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
            if (counts) {
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
                    path_s[__popcll(path & ((1ull << x) - 1))] = t;
                }
                if (__any_sync(full, bad)) r.err = GDN_DEV_BAD_TOKEN;
                r.n_path = __popcll(path);
            }
        }
        if (lane == 0) row_s = r;
    }
    __syncthreads();
    const Row row = row_s;
    const uint16_t *hrow = row.slot >= 0 ? a.history + int64_t(row.slot) * a.h_stride : nullptr;
    const unsigned char *mrow =
        row.mask >= 0 ? reinterpret_cast<const unsigned char *>(a.mask + int64_t(row.mask) * a.mask_stride) : nullptr;
    const uint4 none = make_uint4(0, 0, 0, 0);
    auto history_of = [&](int g) { return hrow ? *reinterpret_cast<const uint4 *>(hrow + int64_t(g) * 8) : none; };
    auto allowed_of = [&](int g) { return mrow ? uint32_t(mrow[g]) : 0xffu; };
    uint4 h[kGroups];
    uint32_t allowed[kGroups];
    if (!row.err) {
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int g = group(k * kThreads + tid);
            const bool there = k * kThreads + tid < locals && g < a.groups;
            h[k] = there ? history_of(g) : none;
            allowed[k] = there ? allowed_of(g) : 0;
        }
    }

    bool bad = false;
    auto touch = [&](int token) {  // marks the group of a token that lies in this slice
        const int g = token >> 3, run = g >> 5;
        if (run % C == rank) atomicOr(mark + (run / C & (kMarkBits / 32 - 1)), 1u << (g & 31));
    };
    if (!row.err) {
        for (int k = tid; k < row.n_path; k += kThreads) touch(path_s[k]);
        for (int k = row.b0 + tid; k < row.b1; k += kThreads) {
            const int t = a.bias_token[k];
            if (t < 0 || t >= a.V || (k > row.b0 && a.bias_token[k - 1] >= t)) bad = true;
            else touch(t);
        }
    }
    const int err = row.err ? row.err : __syncthreads_or(bad) ? GDN_DEV_BAD_TOKEN : 0;  // (row.err is the same for all threads)
    if (err) {
        if (tid == 0 && rank == 0) gdn::record_status(a.status, err);
        cl.barrier_wait(std::move(arrived));
        return;  // the cluster's other CTAs have read the same and leave too
    }

    // x of group g
    auto form = [&](const Raw<T> &in, uint4 h, uint32_t allowed, int local, int g, float (&x)[8]) __attribute__((always_inline)) {
        unpack_raw<T>(in, x);
        uint32_t hw[4] = {h.x, h.y, h.z, h.w};
        const bool marked = (mark[(local >> 5) & (kMarkBits / 32 - 1)] >> (local & 31)) & 1;
        if (marked) {
            for (int k = 0; k < row.n_path; ++k) {
                const int t = path_s[k];
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
    };
    // the groups that registers do not hold
    auto for_rest = [&](auto &&body) {
        if constexpr (kRest) {
#pragma unroll 1
            for (int local = kGroups * kThreads + tid; local < locals; local += kThreads) {
                const int g = group(local);
                if (g >= a.groups) break;
                float x[8];
                form(load_raw<T>(lrow, g), history_of(g), allowed_of(g), local, g, x);
                body(g, x);
            }
        }
    };

    float x[kGroups][8];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const int g = group(k * kThreads + tid);
        if (k * kThreads + tid < locals && g < a.groups) {
            form(raw[k], h[k], allowed[k], k * kThreads + tid, g, x[k]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] = -INFINITY;
        }
    }

    // ---- a warp's maximum; its exponentials and their sum, or the first place of its maximum -----
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, x[k][e]);
    for_rest([&](int, float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, y[e]);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(full, m, o));
    const bool greedy = !(row.t > 0.f);
    // (c is neither 0 nor infinite, and m0 no infinity below, so that x = -inf gives 0; NaN stays NaN)
    const float c = fminf(fmaxf(__fdiv_rn(1.4426950408889634f, row.t), FLT_MIN), FLT_MAX), m0 = m == -INFINITY ? 0.f : m;
    auto weight = [&](float v) { return exp2_fast(__fmul_rn(__fsub_rn(v, m0), c)); };
    Part mine{m, 0.f, INT32_MAX, 0};
    if (greedy) {
        auto look = [&](int g, float (&y)[8]) {
#pragma unroll
            for (int e = 7; e >= 0; --e) {
                if (y[e] == m && m > -INFINITY) mine.best = min(mine.best, 8 * g + e);
                mine.nan |= y[e] != y[e];
            }
        };
#pragma unroll
        for (int k = 0; k < kGroups; ++k) look(group(k * kThreads + tid), x[k]);
        for_rest(look);
        mine.best = __reduce_min_sync(full, mine.best);
        mine.nan = __reduce_or_sync(full, mine.nan);
    } else {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                x[k][e] = weight(x[k][e]);
                x[k][e + 1] = weight(x[k][e + 1]);
                s0 += x[k][e];
                s1 += x[k][e + 1];
            }
        for_rest([&](int, float (&y)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s0 += weight(y[e]);
        });
        mine.sum = gdn::warp_sum(s0 + s1);
    }

    // ---- the row's, from every warp of the cluster in a fixed order ------------------------
    cl.barrier_wait(std::move(arrived));
    if (lane < C) *cl.map_shared_rank(parts + rank * kWarps + warp, lane) = mine;
    cl.sync();
    Part all{-INFINITY, 0.f, INT32_MAX, 0};
    for (int k = lane; k < C * kWarps; k += 32) all.m = fmaxf(all.m, parts[k].m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all.m = fmaxf(all.m, __shfl_xor_sync(full, all.m, o));
    const float M = all.m;
    for (int k = lane; k < C * kWarps; k += 32) {
        const Part q = parts[k];
        if (q.m == M) all.best = min(all.best, q.best);
        all.nan |= q.nan;
        all.sum += q.m == -INFINITY ? q.sum : q.sum * exp2_fast(__fmul_rn(__fsub_rn(q.m, M), c));
    }
    const float total = gdn::warp_sum(all.sum);
    float *prow = a.p + int64_t(n) * a.p_stride;
    auto store = [&](int g, const float (&y)[8]) {
        const int left = a.V - 8 * g;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            if (left >= e + 4) {
                *reinterpret_cast<float4 *>(prow + int64_t(g) * 8 + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            } else {
#pragma unroll
                for (int z = e; z < e + 4; ++z)
                    if (z < left) prow[int64_t(g) * 8 + z] = y[z];
            }
        }
    };
    if (greedy) {
        const int best = __reduce_min_sync(full, all.best), nan = __reduce_or_sync(full, all.nan);
        const float no = nan ? __uint_as_float(0x7fffffffu) : 0.f, yes = nan ? no : 1.f;
        for (int local = tid; local < locals; local += kThreads) {
            const int g = group(local);
            if (g >= a.groups) break;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = 8 * g + e == best ? yes : no;
            store(g, y);
        }
        return;
    }
    // (a NaN total stays; 0: the row has nothing left)
    const float f = total == 0.f ? 0.f : m == -INFINITY ? total * 0.f : exp2_fast(__fmul_rn(__fsub_rn(m, M), c)) / total;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const int g = group(k * kThreads + tid);
        if (k * kThreads + tid < locals && g < a.groups) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[k][e] *= f;
            store(g, x[k]);
        }
    }
    for_rest([&](int g, float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = weight(y[e]) * f;
        store(g, y);
    });
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

// A CTA a sequence, as in the commit itself: a round's few nodes or a prompt's many tokens.
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
            for (int k = tid; k < ns; k += 256) {
                const int t = a.tokens[n0 + k];
                bad |= (!a.accepted || ((path_s >> k) & 1)) && (t < 0 || t >= a.V);
            }
            for (int s2 = tid; s2 < a.S; s2 += 256) dup |= s2 != s && a.slot_map[s2] == slot && commits(a, s2);
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
    for (int k = tid; k < ns; k += 256) {
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
    // A cluster whose registers hold the row, of more CTAs while there are few rows to fill the GPU with.
    int C = 1;
    while (C < kMaxCluster && (int64_t(C) * kSlice < vocab || (rows * 2 * C <= 304 && vocab / (2 * C) >= 2048))) C *= 2;
    a.groups = int((int64_t(vocab) + 7) / 8);
    a.per = ((a.groups + 31) / 32 + C - 1) / C * 32;
    auto k = int64_t(C) * kSlice < vocab ? logits_probs_kernel<T, true> : logits_probs_kernel<T, false>;
    if (C > 8 && cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return GDN_ERR_LAUNCH;
    if (rows * C > INT32_MAX) return GDN_ERR_DIMS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(rows * C));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(C);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
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
    if (gdn::launch_pdl(token_preflight_kernel, dim3(unsigned(S)), dim3(256), 0, st, a) != cudaSuccess) return GDN_ERR_LAUNCH;
    return gdn::launch_pdl(token_commit_kernel, dim3(unsigned(S)), dim3(256), 0, st, a) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
