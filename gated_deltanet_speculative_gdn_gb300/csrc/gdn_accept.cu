// gdn_accept.cu - acceptance of drafted token trees on the device: rejection
// sampling of the draft against the target's probabilities, from given uniforms.
// It takes the place of the host's decision between verify and commit.
//
// Mathematics.  At node t with children x_1, x_2, ... drawn from q without
// replacement, child x (token y) is accepted with probability p'(y) / q'(y), and
// on rejection p' <- norm(max(p' - q', 0)), q' <- norm(q' without y).  Written
// out, every p' along the way is max(p - c q, 0) / W for a number c: with
// p' = max(p - c q, 0) / W and q' = q / Z off the rejected tokens,
//     max(p' - q', 0) = max(p - c q - (W / Z) q, 0) / W,
// since max(max(a, 0) - b, 0) = max(a - b, 0) for b >= 0; and the rejected token
// itself drops out, as u >= (p - c q) Z / (q W) makes p - (c + W / Z) q <= 0.  So
// a rejection costs one sum W = sum_v max(p_v - c q_v, 0) over a row of p and one
// of q and nothing is rewritten, and an accepted first child costs no row at all.
//
// Precision.  The decisions and the place in the cumulative sum stand next to
// borders, so p - c q is formed as an unevaluated pair of floats (Dekker's and
// Knuth's error-free product and sum; c as a pair too) and summed as one: 2^-48
// relative, at ~16 fp32 operations an element, where fp64 arithmetic would run at
// 1/64 of that rate.  A lane's sum is then rounded once to an integer multiple of
// 2^-61 (the sums of a distribution stay below 2): from there on sums, their scans
// and the threshold are 64-bit integers, exact in any order, at two instructions a
// sum.  (As fp64, or as pairs, the reductions and scans of one warp between the
// passes took longer than the passes.)  c, W and Z are pairs.
//
// Mapping.  A cluster of CTAs takes a sequence, each CTA a contiguous slice of
// the vocabulary.  Warp 0 of every CTA walks the tree with the same numbers (so
// the CTAs agree without exchange) and calls for a pass when it needs a sum; a
// pass sums each warp's contiguous range, and the CTAs' sums are exchanged
// through distributed shared memory in rank order.  The last pass's sums are the
// coarse cumulative sum: the CTA and the warp whose range holds the threshold
// narrow it down.  Bound by the latency of the dependent passes (~3 us each at
// 131072 tokens: 1 MB of rows over a cluster, two cluster-wide exchanges): one tree of
// 16 nodes takes 13 us, 64 of them 40 us for 71 MB of rows.
//
// It does not release its dependent kernel early: the commits read `accepted`
// before their own wait.
#include <cooperative_groups.h>

#include <cstdint>

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace {
namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarpsA = kThreads / 32, kMaxCluster = 16;

struct AcceptArgs {
    const float *__restrict__ p, *__restrict__ q;
    int64_t p_stride, q_stride;
    const int32_t *__restrict__ tokens, *__restrict__ parents, *__restrict__ node_off;
    const float *__restrict__ u, *__restrict__ u_next;
    int32_t *accepted, *next_token, *n_accepted, *status;
    int S, N, V, max_nodes, replacement;
};

// An unevaluated sum of two floats, |l| <= ulp(h) / 2 where it is said to be normal.
struct Pair {
    float h, l;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ Pair normal(float h, float l) {  // |h| >= |l|
    const float s = __fadd_rn(h, l);
    return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
// max(p - (ch + cl) q, 0) as a pair
__device__ __forceinline__ Pair residual(float p, float q, float ch, float cl) {
    const float ph = __fmul_rn(ch, q), pl = __fmaf_rn(ch, q, -ph);
    const Pair s = two_sum(p, -ph);
    const float l = __fsub_rn(s.l, __fmaf_rn(cl, q, pl));
    const float h = __fadd_rn(s.h, l);
    if (!(h > 0.f)) return {0.f, 0.f};
    return {h, __fsub_rn(l, __fsub_rn(h, s.h))};
}
// acc += v for terms >= 0; the result is made normal once, at the end of a sum
__device__ __forceinline__ void add(Pair &acc, const Pair &v) {
    const Pair s = two_sum(acc.h, v.h);
    acc.h = s.h;
    acc.l = __fadd_rn(acc.l, __fadd_rn(s.l, v.l));
}
__device__ __forceinline__ Pair plus(const Pair &a, const Pair &b) {
    Pair s = two_sum(a.h, b.h);
    return normal(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair minus(const Pair &a, const Pair &b) { return plus(a, {-b.h, -b.l}); }
__device__ __forceinline__ Pair times(const Pair &a, const Pair &b) {
    const float p = __fmul_rn(a.h, b.h), e = __fmaf_rn(a.h, b.h, -p);
    return normal(p, __fadd_rn(e, __fmaf_rn(a.h, b.l, __fmul_rn(a.l, b.h))));
}
__device__ __forceinline__ Pair over(const Pair &a, const Pair &b) {
    const float q1 = __fdiv_rn(a.h, b.h);
    Pair r = minus(a, times(b, {q1, 0.f}));
    const float q2 = __fdiv_rn(r.h, b.h);
    r = minus(r, times(b, {q2, 0.f}));
    const Pair q = normal(q1, q2);
    return normal(q.h, __fadd_rn(q.l, __fdiv_rn(r.h, b.h)));
}
__device__ __forceinline__ bool less(const Pair &a, const Pair &b) { return a.h < b.h || (a.h == b.h && a.l < b.l); }
__device__ __forceinline__ Pair positive(const Pair &a) { return a.h > 0.f ? a : Pair{0.f, 0.f}; }

// What a pass computes: rows of a node, c, and the tokens that are taken out.
struct Pass {
    const float *p, *q;  // q NULL: the residual is p
    float ch, cl;
    int n_out;
    int last;  // the pass is the one that the next token comes from
};

// The four residuals of vector i of the row (elements 4 i ..; zero past V) from its values.  With q the
// tokens that are taken out have none left by the formula itself.
template <bool kQ>
__device__ __forceinline__ void residual4(const Pass &ps, const int *out, int i, int V, const float4 &p4, const float4 &q4,
                                          Pair (&r)[4]) {
    const float pv[4] = {p4.x, p4.y, p4.z, p4.w}, qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (kQ) r[e] = residual(pv[e], qv[e], ps.ch, ps.cl);
        else r[e] = {pv[e] > 0.f ? pv[e] : 0.f, 0.f};
    }
    if (!kQ) {
        for (int k = 0; k < ps.n_out; ++k)
            if ((out[k] >> 2) == i) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if ((out[k] & 3) == e) r[e] = {0.f, 0.f};
            }
    }
    if (4 * i + 3 >= V) {  // the row's last vector: what lies behind the row is not read as values
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (4 * i + e >= V) r[e] = {0.f, 0.f};
    }
}
__device__ __forceinline__ float4 vec(const float *row, int i) { return __ldg(reinterpret_cast<const float4 *>(row) + i); }

// Sums in units of 2^-61.
typedef long long Fix;
constexpr float kFix = 2305843009213693952.0f;
__device__ __forceinline__ Fix to_fix(const Pair &v) { return __float2ll_rn(v.h * kFix) + __float2ll_rn(v.l * kFix); }
__device__ __forceinline__ Pair to_pair(Fix v) {
    const float h = __ll2float_rn(v);
    return normal(h * (1.0f / kFix), __ll2float_rn(v - __float2ll_rn(h)) * (1.0f / kFix));
}
__device__ __forceinline__ Fix warp_sum(Fix v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum of vectors [lo, hi) of the row, lanes side by side: four vectors a lane are on their way at a time.
template <bool kQ>
__device__ __forceinline__ Fix sum_range_t(const Pass &ps, const int *out, int lo, int hi, int V) {
    constexpr int U = 4;
    Pair acc = {0.f, 0.f};
    for (int i0 = lo + int(threadIdx.x & 31); i0 < hi; i0 += 32 * U) {
        float4 p4[U], q4[U];
#pragma unroll
        for (int z = 0; z < U; ++z) {
            const int i = min(i0 + 32 * z, hi - 1);
            p4[z] = vec(ps.p, i);
            q4[z] = kQ ? vec(ps.q, i) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int z = 0; z < U; ++z) {
            const int i = i0 + 32 * z;
            if (i >= hi) break;
            Pair r[4];
            residual4<kQ>(ps, out, i, V, p4[z], q4[z], r);
#pragma unroll
            for (int e = 0; e < 4; ++e) add(acc, r[e]);
        }
    }
    return warp_sum(to_fix(acc));
}
__device__ __forceinline__ Fix sum_range(const Pass &ps, const int *out, int lo, int hi, int V) {
    return ps.q ? sum_range_t<true>(ps, out, lo, hi, V) : sum_range_t<false>(ps, out, lo, hi, V);
}

// Warp-collective: the first of the parts (lane k holds part k's sum, 0 past the
// last) whose cumulative sum, from b on, passes thr; b becomes the sum before it.
// When none does (u_next at 1, or a row that is no distribution) the last part that
// is not empty, and thr becomes the largest, so that finer selections take the last
// one too.
__device__ __forceinline__ int select_part(Fix v, Fix &b, Fix &thr) {
    const int lane = threadIdx.x & 31;
    Fix inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Fix y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, v > 0 && b + inc > thr);
    const unsigned some = __ballot_sync(0xffffffffu, v > 0);
    const int k = hit ? __ffs(hit) - 1 : some ? 31 - __clz(some) : 0;
    if (!hit) thr = INT64_MAX;
    b += __shfl_sync(0xffffffffu, inc - v, k);
    return k;
}

__global__ void __launch_bounds__(kThreads, 4) tree_accept_kernel(const AcceptArgs a) {
    __shared__ Fix warp_tot[kWarpsA];
    __shared__ Fix cta_tot[2][kMaxCluster];  // [pass parity][rank], written by every CTA of the cluster
    __shared__ int par[gdn::kMaxSeqNodes], tok[gdn::kMaxSeqNodes], out[gdn::kMaxSeqNodes];
    __shared__ float pc[gdn::kMaxSeqNodes], qc[gdn::kMaxSeqNodes], uc[gdn::kMaxSeqNodes];  // p, q at the parent's row
    __shared__ Pass pass_s;
    __shared__ int err_s, step_s;              // what follows the pass: another, the selection, nothing
    __shared__ Fix base_s, thr_s;              // of the selection
    __shared__ int lo_s, hi_s;
    cg::cluster_group cl = cg::this_cluster();
    const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
    const int s = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) err_s = 0;
    __syncthreads();

    // the tree and the drafted tokens' probabilities, all nodes at once
    const int n0 = a.node_off[s], n1 = a.node_off[s + 1], n = n1 - n0;
    if (n0 < 0 || n1 < n0 || n1 > a.N || (s == 0 && n0 != 0) || (s == a.S - 1 && n1 != a.N) || n > a.max_nodes) {
        if (tid == 0) err_s = GDN_DEV_BAD_NODE_OFF;
    } else if (tid < n) {
        const int p = a.parents[n0 + tid];
        par[tid] = p;
        if (p >= tid || (tid == 0 ? p != -1 : p < 0)) atomicCAS(&err_s, 0, GDN_DEV_BAD_PARENT);
    }
    gdn::grid_dep_wait();  // the drafted tokens, the rows and the uniforms may come from kernels before this one
    __syncthreads();
    const bool tree_ok = err_s == 0;
    __syncthreads();
    if (tree_ok && tid > 0 && tid < n) {
        const int y = a.tokens[n0 + tid];
        tok[tid] = y;
        uc[tid] = a.u[n0 + tid];
        if (y < 0 || y >= a.V) {
            atomicCAS(&err_s, 0, GDN_DEV_BAD_TOKEN);
        } else {
            const int64_t row = n0 + par[tid];
            pc[tid] = a.p[row * a.p_stride + y];
            qc[tid] = a.q ? a.q[row * a.q_stride + y] : 1.f;
        }
    }
    cl.sync();  // also: every CTA of the cluster runs before another writes its shared memory
    if (err_s || n == 0) {  // the whole cluster: every CTA has found the same
        if (rank == 0 && tid == 0) {
            if (err_s) gdn::record_status(a.status, err_s);
            a.accepted[s] = -1;
            a.next_token[s] = -1;
            a.n_accepted[s] = 0;
        }
        return;
    }

    // vectors of the row: CTA `rank` takes [v0, v1), its warp w [w0, w1), in order
    const int nvec = (a.V + 3) / 4;
    const int per = (nvec + C - 1) / C, v0 = min(nvec, rank * per), v1 = min(nvec, v0 + per);
    const int perw = (v1 - v0 + kWarpsA - 1) / kWarpsA, w0 = min(v1, v0 + warp * perw), w1 = min(v1, w0 + perw);

    // warp 0's walk, the same in every lane; lane l looks after the parents of nodes l and l + 32
    int cur = 0, t = 1, depth = 1, n_out = 0, parity = 0;  // t: the first node that has not been looked at
    Pair c = {0.f, 0.f}, W = {1.f, 0.f}, Z = {1.f, 0.f};
    bool fallback = false;
    Pass ps;
    const float un = a.u_next[s];
    const int par_lo = lane < n ? par[lane] : -2, par_hi = lane + 32 < n ? par[lane + 32] : -2;
    auto kids_from = [&](int node, int first) {  // node's children from `first` on, as a mask
        const unsigned long long m = (static_cast<unsigned long long>(__ballot_sync(0xffffffffu, par_hi == node)) << 32) |
                                     __ballot_sync(0xffffffffu, par_lo == node);
        return first < 64 ? m >> first << first : 0ull;
    };
    for (;;) {
        if (warp == 0) {
            bool need = false;
            unsigned long long kids = kids_from(cur, t);
            while (kids && Z.h > 0.f && !need) {
                const int x = __ffsll(static_cast<long long>(kids)) - 1, y = tok[x];
                kids &= kids - 1;
                t = x + 1;
                bool was_out = false;
                for (int k = 0; k < n_out; ++k) was_out |= out[k] == y;
                const float qx = was_out && a.q ? 0.f : qc[x];
                Pair px = {0.f, 0.f};
                if (!was_out) px = a.q ? positive(minus({pc[x], 0.f}, times(c, {qx, 0.f}))) : positive({pc[x], 0.f});
                // both sides times 2^64 (exact): the low parts of small probabilities stay normal
                constexpr float kUp = 18446744073709551616.0f;
                if (less(times(times({uc[x], 0.f}, {qx * kUp, 0.f}), W), times({px.h * kUp, px.l * kUp}, Z))) {
                    cur = x;
                    ++depth;
                    n_out = 0;
                    c = {0.f, 0.f};
                    W = Z = {1.f, 0.f};
                    kids = kids_from(cur, t);
                } else {
                    if (!(a.q && a.replacement) && !was_out) {
                        __syncwarp();
                        if (lane == 0) out[n_out] = y;
                        __syncwarp();
                        ++n_out;
                    }
                    if (a.q) {
                        c = plus(c, over(W, Z));
                        if (!a.replacement) Z = positive(minus(Z, {qx, 0.f}));
                        need = kids && Z.h > 0.f;  // the sum is wanted only if another child is tried
                    } else {
                        W = positive(minus(W, px));
                    }
                }
            }
            if (lane == 0) {
                const int64_t row = n0 + cur;
                pass_s.p = a.p + row * a.p_stride;
                pass_s.q = a.q && c.h > 0.f && !fallback ? a.q + row * a.q_stride : nullptr;
                pass_s.ch = c.h;
                pass_s.cl = c.l;
                pass_s.n_out = fallback || a.q ? 0 : n_out;
                pass_s.last = !need;
            }
        }
        __syncthreads();
        ps = pass_s;
        const Fix wt = sum_range(ps, out, w0, w1, a.V);
        if (lane == 0) warp_tot[warp] = wt;
        __syncthreads();
        if (warp == 0) {
            const Fix v = warp_sum(lane < kWarpsA ? warp_tot[lane] : 0);
            if (lane < C) cl.map_shared_rank(&cta_tot[0][0], lane)[parity * kMaxCluster + rank] = v;
        }
        cl.sync();
        if (warp == 0) {
            const Fix mine = lane < C ? cta_tot[parity][lane] : 0;
            const Fix total = warp_sum(mine);
            int step = 0;
            if (ps.last) {
                if (total <= 0 && !fallback) {
                    fallback = true;  // nothing is left: the target's own row
                } else {
                    // cumulative sums pass u total exactly where they pass its floor; u in units of 2^-63
                    const unsigned long long u63 = __float2ull_rn(fminf(fmaxf(un, 0.f), 1.f) * 9223372036854775808.0f);
                    Fix b = 0, thr = Fix(__umul64hi(u63, static_cast<unsigned long long>(max(total, Fix(0))) << 1));
                    const bool owner = select_part(mine, b, thr) == rank;
                    step = owner ? 2 : 1;
                    if (owner) {
                        const int k = select_part(lane < kWarpsA ? warp_tot[lane] : 0, b, thr);
                        if (lane == 0) {
                            base_s = b;
                            thr_s = thr;
                            lo_s = min(v1, v0 + k * perw);
                            hi_s = min(v1, v0 + (k + 1) * perw);
                        }
                    }
                }
            }
            if (!step) W = to_pair(total);
            if (lane == 0) step_s = step;
        }
        parity ^= 1;
        __syncthreads();
        if (step_s) break;
    }

    // ---- the next token: the owner narrows its warp's range down to 32 vectors
    if (rank == 0 && tid == 0) {
        a.accepted[s] = cur;
        a.n_accepted[s] = depth;
    }
    if (step_s != 2) return;
    while (hi_s - lo_s > 32) {
        const int lo = lo_s, hi = hi_s, part = (hi - lo + kWarpsA - 1) / kWarpsA;
        const Fix wt = sum_range(ps, out, min(hi, lo + warp * part), min(hi, lo + (warp + 1) * part), a.V);
        if (lane == 0) warp_tot[warp] = wt;
        __syncthreads();
        if (warp == 0) {
            Fix b = base_s, thr = thr_s;
            const int k = select_part(lane < kWarpsA ? warp_tot[lane] : 0, b, thr);
            if (lane == 0) {
                base_s = b;
                thr_s = thr;
                lo_s = min(hi, lo + k * part);
                hi_s = min(hi, lo + (k + 1) * part);
            }
        }
        __syncthreads();
    }
    if (warp == 0) {
        Pair r[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
        const int i = lo_s + lane;
        if (i < hi_s) {
            if (ps.q) residual4<true>(ps, out, i, a.V, vec(ps.p, i), vec(ps.q, i), r);
            else residual4<false>(ps, out, i, a.V, vec(ps.p, i), make_float4(0.f, 0.f, 0.f, 0.f), r);
        }
        Fix e[4], run = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            run += to_fix(r[k]);
            e[k] = run;
        }
        Fix b = base_s, thr = thr_s;
        const int src = select_part(run, b, thr);
        if (lane == src) {
            // the first that passes the threshold, else the last that is not 0
            int k = e[3] > e[2] ? 3 : e[2] > e[1] ? 2 : e[1] > e[0] ? 1 : 0;
#pragma unroll
            for (int z = 3; z >= 0; --z)
                if (e[z] > (z ? e[z - 1] : 0) && b + e[z] > thr) k = z;
            a.next_token[s] = min(max(4 * i + k, 0), a.V - 1);
        }
    }
}

}  // namespace

extern "C" int gdn_tree_accept(const gdn_dims *dims, int vocab, const float *p, int64_t p_stride, const float *q,
                               int64_t q_stride, int replacement, const int32_t *tokens, const int32_t *parents,
                               const int32_t *node_off, const float *u, const float *u_next, int32_t *accepted,
                               int32_t *next_token, int32_t *n_accepted, int32_t *status, void *stream) {
    int rc = gdn::check_dims(dims);
    if (rc) return rc;
    if (!status) return GDN_ERR_NULL;
    if (vocab < 1 || vocab > (1 << 28) || (replacement != 0 && replacement != 1)) return GDN_ERR_ARG;
    const int64_t S = dims->n_seqs, N = dims->n_nodes;
    if (S == 0) return GDN_OK;
    if (!node_off || !accepted || !next_token || !n_accepted || !u_next ||
        (N > 0 && (!p || !tokens || !parents || !u)))
        return GDN_ERR_NULL;
    const int64_t row = (int64_t(vocab) + 3) / 4 * 4;
    if (N > 0 && (p_stride < row || p_stride % 4 || (q && (q_stride < row || q_stride % 4)))) return GDN_ERR_STRIDE;
    if (!gdn::aligned16(p) || !gdn::aligned16(q)) return GDN_ERR_ALIGN;
    const gdn::Span outs[] = {{accepted, size_t(S * 4)}, {next_token, size_t(S * 4)}, {n_accepted, size_t(S * 4)}};
    const gdn::Span ins[] = {{p, gdn::strided_bytes(N, p_stride, row)},
                             {q, gdn::strided_bytes(N, q_stride, row)},
                             {tokens, size_t(N * 4)},
                             {parents, size_t(N * 4)},
                             {node_off, size_t((S + 1) * 4)},
                             {u, size_t(N * 4)},
                             {u_next, size_t(S * 4)},
                             {status, 4}};
    if ((rc = gdn::check_alias(outs, 3, ins, 8))) return rc;

    AcceptArgs a{p, q, p_stride, q_stride, tokens, parents, node_off, u, u_next, accepted, next_token, n_accepted,
                 status, int(S), int(N), vocab, dims->max_seq_nodes, replacement};
    // A cluster as large as leaves every CTA resident at once (four of 256 threads per SM) and a slice of one
    // vector a thread.  64 sequences of 131072 tokens, three sets of rows in turn: 40 us with 8 CTAs each, 45 us
    // with 4 of 512 threads; one sequence 12.9 us with 16, 16.2 with 8 of 512.  (More CTAs than are resident at
    // once: 48 us, the second wave runs alone.)
    int C = 1;
    while (C < kMaxCluster && int64_t(vocab) / (2 * C) >= 1024 && S * 2 * C <= 608) C *= 2;
    if (C > 8 && cudaFuncSetAttribute(tree_accept_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return GDN_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(S * C));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(C);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, tree_accept_kernel, a) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}
