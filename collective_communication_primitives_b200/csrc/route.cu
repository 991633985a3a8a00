// Router of a mixture-of-experts layer: softmax over the experts' scores, the k best, their weights; and
// the gradient of the scores.
//
//   P = softmax(x[t]),  idx[t][s] = the s-th largest score (the lower id among equals),
//   w[t][s] = P[idx[t][s]], or with `normalise` P[idx[t][s]] / sum over the picked ones
//   gradient, from g = dL/dw:
//     normalise:  dx[e] = sum over s with idx[s] = e of w[s] (g[s] - sum_q g[q] w[q])
//     otherwise:  dx[e] = P[e] (G[e] - sum_q g[q] w[q]),  G[e] = the sum of g[s] over s with idx[s] = e
//
// One pass: a token's row is held in the registers of a group of lanes (8 scores per lane up to 256
// experts, so that a warp takes 32 / lanes tokens and a lane's row piece is one or two 16-byte loads) as
// order-preserving integers, which each lane sorts (a network: 19 exchanges of 8). A round of "largest that is
// left" is then the group's maximum over the lanes' first ones, and one lane that moves up. bf16 scores leave
// room for the id in the integer; for fp32 the ids of all picks are looked up at the end, side by side. The
// sum over the whole row is formed only where the weights are shares of it. What bounds it with many tokens is
// instructions, integer ones before all (issue slots 85 to 93% busy, the integer pipe 62 to 75%, 6 to 7 warps ready on
// a scheduler); with few the launch; the gradient waits for its loads (61% and 48%). Rows of more than 1024 experts are read again for every round, a warp per token
// (from cache; a row is at most 16 KiB). Measured on B200, kernels alone: 8 ranks x 8192 tokens x 64 experts bf16,
// k = 2, 10.3 us (the bytes take 1.5 at the copy rate), the gradient 14.4; 4 x 4099 x 256 fp32, k = 8, 15.7 us and
// 14.3 (8.1 in all); one token 4.1 us; 4096 x 2048 fp32, k = 8, 69 us, the gradient 35 to 37.
// Scores that are NaN are picked last and make the row's weights NaN; a row of nothing but -inf has
// weight 0 for every pick.
#include <algorithm>

#include "common.cuh"

namespace simcomm {

constexpr int kRouteThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Unsigned integers in the order of the floats, NaN below everything, 0 below that (no score).
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 and +0 are equal scores
    const uint32_t o = u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
    return x != x ? 1u : o;
}

template <int DT> __device__ __forceinline__ float ld_score(const void* row, int e) { return load_elem<DT>(row, size_t(e)); }

// The VPL scores from e0 of a row of E (missing ones: `fill`). vec: 16-byte loads, E a multiple of 8.
template <int DT, int VPL>
__device__ __forceinline__ void ld_scores(float (&v)[VPL], const void* row, int e0, int E, bool vec, float fill) {
    if (vec) {
        using P = Pack16<DT>;
#pragma unroll
        for (int j = 0; j < VPL; j += P::L) {
            float part[P::L];
            if (e0 + j < E) {
                P::unpack(ld_stream_v4(static_cast<const char*>(row) + size_t(e0 + j) * Elem<DT>::kBytes), part);
            } else {
#pragma unroll
                for (int q = 0; q < P::L; ++q) part[q] = fill;
            }
#pragma unroll
            for (int q = 0; q < P::L; ++q) v[j + q] = part[q];
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) v[j] = e0 + j < E ? ld_score<DT>(row, e0 + j) : fill;
    }
}

template <int LPT> __device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}
template <int LPT> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
template <int LPT> __device__ __forceinline__ uint32_t group_umax(uint32_t v) {
    if constexpr (LPT == 32) {
        return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int d = LPT / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    }
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// The row's maximum over the group, NaN if any score is.
template <int LPT, int VPL> __device__ __forceinline__ float row_max(const float (&v)[VPL]) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) m = max_nan(m, v[j]);
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

// Sorts a lane's integers, largest first: Batcher's odd-even merge network.
template <int N> __device__ __forceinline__ void sort_down(uint32_t (&x)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t a = x[i + j], b = x[i + j + k];
                        x[i + j] = max(a, b);
                        x[i + j + k] = min(a, b);
                    }
}

// Softmax terms of the row in place: v[j] = e^(v[j] - max), the sum over the group returned. Missing
// scores are -inf. A row of nothing but -inf has terms and sum 0; NaN or +inf makes the sum NaN.
template <int LPT, int VPL> __device__ __forceinline__ float softmax_terms(float (&v)[VPL], float* top) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) m = fmaxf(m, v[j]);
    m = group_max<LPT>(m);
    *top = m;
    const float base = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        v[j] = exp2_fast((v[j] - base) * kLog2e);
        sum += v[j];
    }
    return group_sum<LPT>(sum);
}

// A warp's tokens (of one rank: blockIdx.y) and their picks. Picks of consecutive tokens lie together in
// memory, so a warp's are moved by all its lanes at once, through shared memory.
template <int LPT> struct RouteWarp {
    static constexpr int kTokens = 32 / LPT;
    int lane, sub, grp, rank;
    uint32_t first, t;  // the warp's first token, the group's
    int count;          // tokens of the warp
    bool live;

    __device__ __forceinline__ RouteWarp(const RouteArgs& a) {
        lane = threadIdx.x & 31;
        sub = lane % LPT;
        grp = lane / LPT;
        rank = a.rank0 + int(blockIdx.y);
        const uint32_t T = uint32_t(a.T);  // tokens * k fits 31 bits
        first = (blockIdx.x * (kRouteThreads / 32) + (threadIdx.x >> 5)) * kTokens;  // below T + a CTA: 32 bits hold it
        t = first + grp;
        count = first < T ? int(min(uint32_t(kTokens), T - first)) : 0;
        live = t < T;
    }
    __device__ __forceinline__ size_t pick0(const RouteArgs& a) const { return size_t(first) * a.k; }
};

// The score that an order key stands for (any NaN for a NaN's).
__device__ __forceinline__ float key_score(uint32_t o) {
    return o == 1u ? __int_as_float(0x7fffffff) : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

template <int DT, int LPT, int VPL>
__global__ void __launch_bounds__(kRouteThreads) k_route(const __grid_constant__ RouteArgs a) {
    // [warps][ids, terms][tokens of a warp][k], then for fp32 [warps][32 VPL] the keys as they came
    extern __shared__ __align__(16) uint32_t s_picks[];
    if (status_failed(a.ctl)) return;
    const RouteWarp<LPT> w(a);
    const unsigned gmask = LPT == 32 ? 0xffffffffu : ((1u << (LPT & 31)) - 1u) << (w.grp * LPT);
    const char* row = static_cast<const char*>(a.logits[w.rank]) + size_t(w.live ? w.t : 0) * a.E * Elem<DT>::kBytes;
    const int e0 = w.sub * VPL, warp = threadIdx.x >> 5;
    constexpr bool kPacked = DT == COLL_BF16;
    float v[VPL];
    ld_scores<DT, VPL>(v, row, e0, w.live ? a.E : 0, a.vec, -INFINITY);
    const float top = row_max<LPT, VPL>(v);
    const bool nan = top != top;
    uint32_t key[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const uint32_t u = __float_as_uint(v[j] + 0.0f);  // -0 and +0 are equal scores
        key[j] = u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
    }
    if (__any_sync(0xffffffffu, nan)) {  // a NaN comes behind every number
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (v[j] != v[j]) key[j] = kPacked ? 0x10000u : 1u;
    }
    if constexpr (kPacked) {  // the upper half the score's order, the lower the id's complement
#pragma unroll
        for (int j = 0; j < VPL; ++j) key[j] = (key[j] & 0xffff0000u) | uint32_t(0xffff - (e0 + j));
    }
    if (e0 + VPL > a.E) {  // missing scores: below everything
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (e0 + j >= a.E) key[j] = 0u;
    }
    const int n = w.kTokens * a.k;
    uint32_t* all_ids = s_picks + warp * 2 * n;
    uint32_t* all_terms = all_ids + n;
    uint32_t* ids = all_ids + w.grp * a.k;
    uint32_t* terms = all_terms + w.grp * a.k;
    uint32_t* kept = s_picks + (kRouteThreads / 32) * 2 * ((n + 1) / 2 * 2) + warp * 32 * VPL;
    if constexpr (!kPacked) {
#pragma unroll
        for (int j = 0; j < VPL; j += 2) *reinterpret_cast<uint2*>(kept + w.lane * VPL + j) = make_uint2(key[j], key[j + 1]);
    }
    sort_down<VPL>(key);
    for (int s = 0; s < a.k; ++s) {
        const uint32_t all = group_umax<LPT>(key[0]);
        bool mine = key[0] == all;
        if constexpr (!kPacked) mine = w.lane == __ffs(__ballot_sync(0xffffffffu, mine) & gmask) - 1;
        if (mine) {  // one lane of the group moves up
#pragma unroll
            for (int j = 0; j + 1 < VPL; ++j) key[j] = key[j + 1];
            key[VPL - 1] = 0u;
            ids[s] = uint32_t(w.sub);
            terms[s] = all;
        }
    }
    __syncwarp();
    // side by side: the picks' ids and terms, e^(score - max)
    const float base = top == -INFINITY ? 0.0f : top;
    float picked = 0.0f;
    constexpr int kTurns = (32 + LPT - 1) / LPT;  // of a lane over its group's picks, k <= 32
    uint32_t id[kTurns];
    float term[kTurns];
#pragma unroll
    for (int q = 0; q < kTurns; ++q) {
        const int s = w.sub + q * LPT;
        if (s >= a.k) break;
        const uint32_t o = terms[s];
        if constexpr (kPacked) {
            id[q] = 0xffffu - (o & 0xffffu);
            const uint32_t u = o & 0xffff0000u;  // a negative score's complement has zeros below
            term[q] = exp2_fast((key_score(u == 0x10000u ? 1u : u & 0x80000000u ? u : u | 0xffffu) - base) * kLog2e);
        } else {
            const uint32_t sub = ids[s];
            int before = 0;  // equal scores of the same lane that were picked earlier
            for (int r = 0; r < s; ++r) before += terms[r] == o && ids[r] == sub;
            const uint32_t* from = kept + (w.grp * LPT + sub) * VPL;
            int at = 0;
            int seen = 0;
            for (int j = 0; j < VPL; ++j)
                if (from[j] == o) {
                    if (seen == before) at = j;
                    ++seen;
                }
            id[q] = sub * VPL + at;
            term[q] = exp2_fast((key_score(o) - base) * kLog2e);
        }
        picked += term[q];
    }
    float total;
    if (a.normalise) {
        total = group_sum<LPT>(picked);
        if (nan) total = top;  // NaN anywhere in the row reaches every weight; of +inf, inf - inf does
    } else {
        float unused;
        total = softmax_terms<LPT, VPL>(v, &unused);
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < kTurns; ++q) {
        const int s = w.sub + q * LPT;
        if (s >= a.k) break;
        ids[s] = id[q];
        terms[s] = __float_as_uint(total == 0.0f ? 0.0f : term[q] / total);
    }
    __syncwarp();
    for (int i = w.lane; i < w.count * a.k; i += 32) {
        a.idx_out[w.rank][w.pick0(a) + i] = int32_t(all_ids[i]);
        a.weight[w.rank][w.pick0(a) + i] = __uint_as_float(all_terms[i]);
    }
}

// row[ids[s]] += value(s) for the group's k picks; a pick that shares its id with another of the same turn goes
// after it, in order. Warp-collective (every group has the same `most`).
template <int LPT, typename Value>
__device__ __forceinline__ void add_picks(const RouteWarp<LPT>& w, float* row, const uint32_t* ids, int k, int most, Value value) {
    for (int s0 = 0; s0 < most; s0 += LPT) {
        const int s = s0 + w.sub;
        const bool in = s < k;
        const uint32_t id = in ? ids[s] : 0u;
        const float x = in ? value(s) : 0.0f;
        // lanes without a pick stand alone
        const unsigned same = __match_any_sync(0xffffffffu, in ? id << 5 | uint32_t(w.grp) : 0x80000000u | uint32_t(w.lane));
        const int turn = __popc(same & ((1u << w.lane) - 1u));
        for (int t = 0; __any_sync(0xffffffffu, in && turn >= t); ++t) {
            if (in && turn == t) row[id] += x;
            __syncwarp();
        }
    }
}

template <int DT, int LPT, int VPL>
__global__ void __launch_bounds__(kRouteThreads) k_route_grad(const __grid_constant__ RouteArgs a) {
    // [warps][32 VPL] a number per score of the warp's tokens, then [warps][ids, g, score][tokens of a warp][k]
    extern __shared__ __align__(16) uint32_t s_grad[];
    if (status_failed(a.ctl)) return;
    const RouteWarp<LPT> w(a);
    const char* row = static_cast<const char*>(a.logits[w.rank]) + size_t(w.live ? w.t : 0) * a.E * Elem<DT>::kBytes;
    const int e0 = w.sub * VPL, warp = threadIdx.x >> 5;
    float v[VPL];
    ld_scores<DT, VPL>(v, row, e0, w.live ? a.E : 0, a.vec, -INFINITY);
    float* slots = reinterpret_cast<float*>(s_grad) + warp * 32 * VPL;  // scores of the group: [LPT * VPL]
    const int n = w.kTokens * a.k;
    uint32_t* ids_all = s_grad + kRouteThreads * VPL + warp * 3 * n;
    float* g_all = reinterpret_cast<float*>(ids_all + n);
    float* x_all = g_all + n;
    bool bad = false;
    for (int i = w.lane; i < w.count * a.k; i += 32) {
        const int e = a.idx_in[w.rank][w.pick0(a) + i];
        const bool ok = e >= 0 && e < a.E;
        bad = bad || !ok;
        ids_all[i] = ok ? uint32_t(e) : 0u;
        g_all[i] = ok ? a.grad_weight[w.rank][w.pick0(a) + i] : 0.0f;
        if (a.normalise)
            x_all[i] = ld_score<DT>(static_cast<const char*>(a.logits[w.rank]) + size_t(w.first + i / a.k) * a.E * Elem<DT>::kBytes, ok ? e : 0);
    }
    if (bad) raise_status(a.ctl, COLL_ERR_INVALID_ARG);
#pragma unroll
    for (int j = 0; j < VPL; j += 4) *reinterpret_cast<float4*>(slots + w.lane * VPL + j) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncwarp();
    const uint32_t* ids = ids_all + w.grp * a.k;
    const float* gw = g_all + w.grp * a.k;
    float* xs = x_all + w.grp * a.k;
    float* mine = slots + w.grp * LPT * VPL;
    const int k = w.live ? a.k : 0;
    float G[VPL];
    if (a.normalise) {
        // only the picked scores matter: w[s] = term[s] / total, dx = sum of w (g - sum_q g w); but the forward pass's
        // weights are NaN where any score of the row is
        const float all = row_max<LPT, VPL>(v);
        float top = -INFINITY;
        for (int s = w.sub; s < k; s += LPT) top = fmaxf(top, xs[s]);
        top = group_max<LPT>(top);  // a NaN comes through by its own term
        const float base = top == -INFINITY ? 0.0f : top;
        float total = 0.0f, dot = 0.0f;
        for (int s = w.sub; s < k; s += LPT) {
            const float term = exp2_fast((xs[s] - base) * kLog2e);
            xs[s] = term;
            total += term;
            dot = __fmaf_rn(gw[s], term, dot);
        }
        total = group_sum<LPT>(total);  // by all lanes, before rows part company
        dot = group_sum<LPT>(dot);
        if (all != all) total = all;
        const float inv = total == 0.0f ? 0.0f : 1.0f / total, mean = dot * inv;
        __syncwarp();
        add_picks<LPT>(w, mine, ids, k, a.k, [&](int s) { return xs[s] * inv * (gw[s] - mean); });
#pragma unroll
        for (int j = 0; j < VPL; ++j) G[j] = slots[w.lane * VPL + j];
    } else {
        float top;
        const float total = softmax_terms<LPT, VPL>(v, &top);
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        add_picks<LPT>(w, mine, ids, k, a.k, [&](int s) { return gw[s]; });
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            G[j] = slots[w.lane * VPL + j];
            dot = __fmaf_rn(G[j], v[j], dot);
        }
        const float mean = group_sum<LPT>(dot) * inv;
#pragma unroll
        for (int j = 0; j < VPL; ++j) G[j] = v[j] * inv * (G[j] - mean);
    }
    if (!w.live) return;
    char* out = static_cast<char*>(a.grad_logits[w.rank]) + size_t(w.t) * a.E * Elem<DT>::kBytes;
    if (a.vec) {
        using P = Pack16<DT>;
#pragma unroll
        for (int j = 0; j < VPL; j += P::L) {
            if (e0 + j >= a.E) continue;
            float part[P::L];
#pragma unroll
            for (int q = 0; q < P::L; ++q) part[q] = G[j + q];
            st_v4(out + size_t(e0 + j) * Elem<DT>::kBytes, P::pack(part));
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (e0 + j < a.E) store_elem<DT>(out, size_t(e0 + j), G[j]);
    }
}

// More than 1024 experts: a warp per token, the row read again for every round.
template <int DT> __global__ void __launch_bounds__(kRouteThreads) k_route_wide(const __grid_constant__ RouteArgs a, int backward) {
    if (status_failed(a.ctl)) return;
    const int lane = threadIdx.x & 31;
    const size_t t = size_t(blockIdx.x) * (kRouteThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int rank = a.rank0 + int(blockIdx.y);
    const void* row = static_cast<const char*>(a.logits[rank]) + t * a.E * Elem<DT>::kBytes;
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, ld_score<DT>(row, e));
    m = group_max<32>(m);
    const float base = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f;
    for (int e = lane; e < a.E; e += 32) sum += exp2_fast((ld_score<DT>(row, e) - base) * kLog2e);
    sum = group_sum<32>(sum);
    if (!backward) {
        uint32_t last = 0xffffffffu;  // the last pick: (order key, id), picks go down the keys and up the ids
        int last_e = -1;
        float picked = 0.0f;
        for (int s = 0; s < a.k; ++s) {
            uint32_t best = 0u;
            int at = INT32_MAX;
            for (int e = lane; e < a.E; e += 32) {
                const uint32_t key = order_key(ld_score<DT>(row, e));
                const bool left = key < last || (key == last && e > last_e);
                if (left && key > best) {
                    best = key;
                    at = e;
                }
            }
            const uint32_t all = __reduce_max_sync(0xffffffffu, best);
            const int e = int(__reduce_min_sync(0xffffffffu, best == all ? unsigned(at) : unsigned(INT32_MAX)));
            last = all;
            last_e = e;
            const float term = exp2_fast((ld_score<DT>(row, e) - base) * kLog2e);
            picked += term;
            if (lane == 0) {
                a.idx_out[rank][t * a.k + s] = e;
                a.weight[rank][t * a.k + s] = term;
            }
        }
        if (lane == 0) {
            const float total = a.normalise ? picked + 0.0f * sum : sum;
            for (int s = 0; s < a.k; ++s) {
                float* w = a.weight[rank] + t * a.k + s;
                *w = total == 0.0f ? 0.0f : *w / total;
            }
        }
        return;
    }
    const int32_t* idx = a.idx_in[rank] + t * a.k;
    const float* gw = a.grad_weight[rank] + t * a.k;
    bool bad = false;
    float top = -INFINITY;
    for (int s = 0; s < a.k; ++s) {
        if (idx[s] < 0 || idx[s] >= a.E) {
            bad = true;
            continue;
        }
        const float x = ld_score<DT>(row, idx[s]);
        top = x > top || x != x ? x : top;
    }
    if (bad) {  // nothing written: the call has failed
        if (lane == 0) raise_status(a.ctl, COLL_ERR_INVALID_ARG);
        return;
    }
    const float from = a.normalise ? (top == -INFINITY ? 0.0f : top) : base;
    float total = 0.0f, dot = 0.0f;
    for (int s = 0; s < a.k; ++s) {
        const float term = exp2_fast((ld_score<DT>(row, idx[s]) - from) * kLog2e);
        total += term;
        dot = __fmaf_rn(gw[s], term, dot);
    }
    total = a.normalise ? total + 0.0f * sum : sum;  // a NaN anywhere in the row reaches every pick
    const float inv = total == 0.0f ? 0.0f : 1.0f / total, mean = dot * inv;
    for (int e = lane; e < a.E; e += 32) {
        float g = 0.0f;
        int hits = 0;
        for (int s = 0; s < a.k; ++s)
            if (idx[s] == e) {
                g += gw[s];
                ++hits;
            }
        float d = 0.0f;
        if (!a.normalise) d = exp2_fast((ld_score<DT>(row, e) - from) * kLog2e) * inv * (g - mean);
        else if (hits) d = exp2_fast((ld_score<DT>(row, e) - from) * kLog2e) * inv * (g - float(hits) * mean);
        store_elem<DT>(static_cast<char*>(a.grad_logits[rank]) + t * a.E * Elem<DT>::kBytes, size_t(e), d);
    }
}

template <int DT> static cudaError_t launch_route_dt(const RouteArgs& a, bool backward, cudaStream_t s) {
    auto grid = [&](int lanes) {
        const size_t per_cta = size_t(kRouteThreads / lanes);
        return dim3(unsigned((a.T + per_cta - 1) / per_cta), unsigned(a.ranks));
    };
#define SIMCOMM_ROUTE(LPT, VPL)                                                                              \
    do {                                                                                                     \
        const size_t picks = size_t(kRouteThreads / LPT) * a.k * 4;                                          \
        if (backward) {                                                                                      \
            const size_t smem = size_t(kRouteThreads) * VPL * 4 + 3 * picks;                                 \
            if (smem > 48 * 1024) {                                                                          \
                cudaError_t e = cudaFuncSetAttribute(k_route_grad<DT, LPT, VPL>,                             \
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)); \
                if (e != cudaSuccess) return e;                                                              \
            }                                                                                                \
            k_route_grad<DT, LPT, VPL><<<grid(LPT), kRouteThreads, smem, s>>>(a);                            \
        } else {                                                                                             \
            const size_t kept = DT == COLL_FP32 ? size_t(kRouteThreads) * VPL * 4 : 0;                       \
            const size_t smem = 2 * picks + 64 + kept;                                                       \
            if (smem > 48 * 1024) {                                                                          \
                cudaError_t e = cudaFuncSetAttribute(k_route<DT, LPT, VPL>,                                  \
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)); \
                if (e != cudaSuccess) return e;                                                              \
            }                                                                                                \
            k_route<DT, LPT, VPL><<<grid(LPT), kRouteThreads, smem, s>>>(a);                                 \
        }                                                                                                    \
        return cudaGetLastError();                                                                           \
    } while (0)
    if (a.E <= 8) SIMCOMM_ROUTE(1, 8);
    if (a.E <= 16) SIMCOMM_ROUTE(2, 8);
    if (a.E <= 32) SIMCOMM_ROUTE(4, 8);
    if (a.E <= 64) SIMCOMM_ROUTE(8, 8);
    if (a.E <= 128) SIMCOMM_ROUTE(16, 8);
    if (a.E <= 256) SIMCOMM_ROUTE(32, 8);
    if (a.E <= 512) SIMCOMM_ROUTE(32, 16);
    if (a.E <= 1024) SIMCOMM_ROUTE(32, 32);
#undef SIMCOMM_ROUTE
    k_route_wide<DT><<<grid(32), kRouteThreads, 0, s>>>(a, backward ? 1 : 0);
    return cudaGetLastError();
}

cudaError_t launch_route(const RouteArgs& a, int dtype, bool backward, cudaStream_t s) {
    return dtype == COLL_BF16 ? launch_route_dt<COLL_BF16>(a, backward, s) : launch_route_dt<COLL_FP32>(a, backward, s);
}

}  // namespace simcomm
