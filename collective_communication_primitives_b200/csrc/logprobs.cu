// Log probabilities of given tokens, entropy and top alternatives over a vocabulary whose columns are
// sharded over the ranks, and the gradient of the scores.
//
//   row t's scores x[v], v < V: rank r holds columns [r m, (r+1) m), m = ceil(V / p)
//   M = max x, S = sum e^(x-M), U = sum (x-M) e^(x-M)      (over all ranks: the AllReduce of the rows' statistics)
//   lse = M + ln S,  logprob = x[token] - lse,  entropy = -sum P ln P = ln S - U / S,  P = e^(x - lse)
//   dx[v] = gl ([v = token] - P[v]) - ge P[v] (ln P[v] + entropy),   gl, ge: gradients of logprob and entropy
//
// Forward: one pass over the scores. A thread keeps a running maximum and rescales its sums only when a
// vector of scores brings a larger one; threads, then parts of a row, are joined in a fixed order. Both
// terms of the entropy's form above are non-negative, so nothing cancels. Few rows are cut into parts, one
// CTA each; the last part to finish joins them all. Bound by the scores' bytes, then, for 2-byte scores,
// by the one exponential per score.
//
// Alternatives: each warp keeps its n best as 64-bit keys (the score's order, then the complement of the
// column, so that the lower column wins among equals), one per lane, sorted. A vector whose maximum does
// not pass the n-th key is dismissed by one comparison; the warps of a CTA share the highest n-th score
// found, below which no score can matter.
//
// The exponentials are powers of two, 2^(x log2e - B) with B = M log2e rounded to fp32, so that a score
// costs one fused multiply-add and one ex2: S and U refer to B, and the rounding of B is put back at the
// end (resid below). That holds while |M| is moderate. Masked scores: -inf has probability 0; for the
// arithmetic a score below -2^100 counts as -2^100, which gives it probability 0 next to any score that is
// not masked and keeps 0 * inf out of the sums. A row whose maximum is beyond +-1e5, such as one masked
// throughout by the type's lowest value, is summed again relative to its maximum. A row of nothing but
// -inf has no distribution: lse and logprob -inf, entropy 0, gradient 0. NaN or +inf in a row makes its
// values NaN.
#include <algorithm>

#include "common.cuh"

namespace simcomm {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpUnroll = 4;            // 16-byte loads in flight per thread
constexpr float kLpLog2e = 1.4426950408889634f;
constexpr float kLpLn2 = 0.6931471805599453f;
constexpr float kLpFloor = -0x1p100f;   // scores below count as this in the sums (x log2e is exact at a power of two)
constexpr float kLpFar = 1e5f;          // rows whose maximum is further from 0 are summed again

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Sums of a set of scores relative to its maximum m (at least kLpFloor).
struct Stat {
    float m, s, u;  // s = sum of e, u = sum of e d, over d = x log2e - log2_base(m), e = 2^d
    float raw;      // the maximum before the clamp; NaN if any score is NaN
};
__device__ __forceinline__ Stat stat_none() { return Stat{kLpFloor, 0.0f, 0.0f, -INFINITY}; }
__device__ __forceinline__ float log2_base(float m) { return m * kLpLog2e; }
// Joins b to a: left fold, so the order of calls fixes the rounding.
__device__ __forceinline__ Stat stat_join(const Stat& a, const Stat& b) {
    Stat r;
    r.m = max_nan(a.m, b.m);
    const float base = log2_base(r.m), da = log2_base(a.m) - base, db = log2_base(b.m) - base;
    const float fa = ex2(da), fb = ex2(db);
    r.s = a.s * fa + b.s * fb;
    r.u = __fmaf_rn(a.s * fa, da, a.u * fa) + __fmaf_rn(b.s * fb, db, b.u * fb);
    r.raw = max_nan(a.raw, b.raw);
    return r;
}
__device__ __forceinline__ Stat stat_shfl_xor(const Stat& a, int d) {
    return Stat{__shfl_xor_sync(0xffffffffu, a.m, d), __shfl_xor_sync(0xffffffffu, a.s, d),
                __shfl_xor_sync(0xffffffffu, a.u, d), __shfl_xor_sync(0xffffffffu, a.raw, d)};
}

__device__ __forceinline__ uint32_t score_order(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 and +0 are equal
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_score(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ unsigned long long top_key(float x, uint32_t col) {
    return ((unsigned long long)score_order(x) << 32) | uint32_t(~col);
}

// A warp's n best keys, one per lane, largest in lane 0; nth: the n-th (0 while fewer are held).
struct TopList {
    unsigned long long mine, nth;
    float nth_score;
};

// Takes every lane's key (0: none) into the warp's list; whether the list changed (the same for every lane).
__device__ __forceinline__ bool top_insert(TopList& l, unsigned long long key, int n) {
    const int lane = threadIdx.x & 31;
    bool changed = false;
    unsigned who = __ballot_sync(0xffffffffu, key > l.nth);
    while (who) {
        const int src = __ffs(who) - 1;
        who &= who - 1;
        const unsigned long long k = __shfl_sync(0xffffffffu, key, src);
        if (k <= l.nth) continue;  // the list has risen meanwhile
        const int pos = __popc(__ballot_sync(0xffffffffu, l.mine > k));
        const unsigned long long up = __shfl_up_sync(0xffffffffu, l.mine, 1);
        l.mine = lane < pos ? l.mine : lane == pos ? k : up;
        l.nth = __shfl_sync(0xffffffffu, l.mine, n - 1);
        changed = true;
    }
    return changed;
}

// Offers every lane's `cnt` scores at columns col, col + 1, ... to the warp's list. Warp-collective.
template <int L>
__device__ __forceinline__ void top_offer(TopList& l, const float (&x)[L], int cnt, uint32_t col, int n, uint32_t* s_nth) {
    const int lane = threadIdx.x & 31;
    bool changed = false;
#pragma unroll
    for (int j = 0; j < L; ++j) {
        const unsigned long long key = (j < cnt && x[j] == x[j]) ? top_key(x[j], col + j) : 0ull;
        changed |= top_insert(l, key, n);
    }
    if (changed && l.nth) {
        l.nth_score = order_score(uint32_t(l.nth >> 32));
        if (lane == 0) atomicMax(s_nth, uint32_t(l.nth >> 32));
    }
}

// Adds `x` (missing scores are -inf) to a thread's sums.
template <int L> __device__ __forceinline__ float stat_feed(Stat& st, const float (&x)[L]) {
    float top = x[0];
#pragma unroll
    for (int j = 1; j < L; ++j) top = max_nan(top, x[j]);
    st.raw = max_nan(st.raw, top);
    if (!(top <= st.m)) {  // larger, or NaN
        const float m = top == INFINITY ? __int_as_float(0x7fffffff) : top;
        const float d = log2_base(st.m) - log2_base(m), f = ex2(d);
        st.u = __fmaf_rn(st.s * f, d, st.u * f);
        st.s *= f;
        st.m = m;
    }
    const float base = log2_base(st.m);
#pragma unroll
    for (int j = 0; j < L; ++j) {
        const float d = __fmaf_rn(fmaxf(x[j], kLpFloor), kLpLog2e, -base);
        const float e = ex2(d);
        st.s += e;
        st.u = __fmaf_rn(e, d, st.u);
    }
    return top;
}

template <int DT, bool TOP>
__device__ __forceinline__ void scan_columns(const LogprobArgs& a, size_t row, size_t v0, size_t v1, Stat& st, TopList& l,
                                             uint32_t* s_nth) {
    using P = Pack16<DT>;
    constexpr int L = P::L, D = Elem<DT>::kBytes;
    auto offer = [&](const float (&x)[L], float top, int cnt, uint32_t col) {
        if constexpr (TOP) {
            const bool may = cnt > 0 && (l.nth == 0ull || (top > l.nth_score && score_order(top) >= *(volatile uint32_t*)s_nth) ||
                                         top != top);
            if (__any_sync(0xffffffffu, may)) top_offer<L>(l, x, cnt, col, a.n_top, s_nth);
        }
    };
    for (size_t v = v0; v < v1;) {
        const size_t r = v / a.m, end = min(v1, (r + 1) * a.m);
        const char* base = static_cast<const char*>(a.logits[r]) + (row * a.ld + (v - r * a.m)) * D;
        const size_t n = end - v;
        const size_t head = min(n, size_t((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / D);
        const size_t vecs = (n - head) / L, tail = n - head - vecs * L;
        // less than a vector at either end, one score per lane of the first warp. A warp meets its scores in
        // column order, so a later one that only equals its n-th best does not belong in its list.
        auto ends = [&](size_t from, size_t count) {
            if (count == 0 || threadIdx.x >= 32) return;
            const int cnt = threadIdx.x < count ? 1 : 0;
            float x[L];
#pragma unroll
            for (int j = 0; j < L; ++j) x[j] = -INFINITY;
            if (cnt) x[0] = load_elem<DT>(base, from + threadIdx.x);
            const float top = stat_feed<L>(st, x);
            offer(x, top, cnt, uint32_t(v + from + threadIdx.x));
        };
        ends(0, head);
        const char* body = base + head * D;
        for (size_t i0 = 0; i0 < vecs; i0 += kLpThreads * kLpUnroll) {
            uint4 raw[kLpUnroll];
#pragma unroll
            for (int q = 0; q < kLpUnroll; ++q) {
                const size_t i = i0 + q * kLpThreads + threadIdx.x;
                if (i < vecs) raw[q] = ld_stream_v4(body + i * 16);
            }
#pragma unroll
            for (int q = 0; q < kLpUnroll; ++q) {
                const size_t i = i0 + q * kLpThreads + threadIdx.x;
                if (i0 + q * kLpThreads + (threadIdx.x & ~31u) >= vecs) break;  // none of this warp's
                float x[L];
#pragma unroll
                for (int j = 0; j < L; ++j) x[j] = -INFINITY;
                const int cnt = i < vecs ? L : 0;
                if (cnt) P::unpack(raw[q], x);
                const float top = stat_feed<L>(st, x);
                offer(x, top, cnt, uint32_t(v + head + i * L));
            }
        }
        ends(n - tail, tail);
        v = end;
    }
}

__device__ __forceinline__ float score_at(const LogprobArgs& a, int dtype, size_t row, size_t v) {
    const size_t r = v / a.m, at = row * a.ld + (v - r * a.m);
    return dtype == COLL_BF16 ? load_elem<COLL_BF16>(a.logits[r], at) : load_elem<COLL_FP32>(a.logits[r], at);
}

// The CTA's sum of one float per thread, in a fixed order; the same for every thread.
__device__ __forceinline__ float cta_sum(float v, float* s_w) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < kLpWarps; ++w) t += s_w[w];
    return t;
}

__device__ __forceinline__ float cta_max(float v, float* s_w) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = s_w[0];
    for (int w = 1; w < kLpWarps; ++w) t = max_nan(t, s_w[w]);
    return t;
}

// ln of the sum of e^(x - m) over a row with maximum m, and the row's entropy. CTA-collective.
__device__ __noinline__ float careful_log_sum(const LogprobArgs& a, int dtype, size_t row, float m, float* entropy, float* s_w) {
    float s = 0.0f, u = 0.0f;
    for (size_t v = threadIdx.x; v < a.V; v += kLpThreads) {
        const float d = score_at(a, dtype, row, v) - m, e = expf(d);
        if (e > 0.0f) {
            s += e;
            u = __fmaf_rn(e, d, u);
        }
    }
    s = cta_sum(s, s_w);
    u = cta_sum(u, s_w);
    *entropy = logf(s) - u / s;
    return logf(s);
}

template <int DT, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 4) k_logprobs(const __grid_constant__ LogprobArgs a) {
    __shared__ Stat s_stat[kLpWarps];
    __shared__ unsigned long long s_key[kLpWarps * 32];
    __shared__ float s_w[kLpWarps];
    __shared__ uint32_t s_nth;
    __shared__ int s_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t row = blockIdx.x / a.parts;
    const int part = int(blockIdx.x % a.parts);
    if (threadIdx.x == 0) {
        s_nth = 0u;
        s_flag = status_failed(a.ctl);
    }
    __syncthreads();
    if (s_flag) return;
    const size_t v0 = a.V * part / a.parts, v1 = a.V * (part + 1) / a.parts;
    Stat st = stat_none();
    TopList l{0ull, 0ull, 0.0f};
    scan_columns<DT, TOP>(a, row, v0, v1, st, l, &s_nth);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Stat o = stat_shfl_xor(st, d);
        st = (lane & d) ? stat_join(o, st) : stat_join(st, o);  // lower lane first: the same on both sides
    }
    if (lane == 0) s_stat[warp] = st;
    if constexpr (TOP)
        if (lane < a.n_top) s_key[warp * a.n_top + lane] = l.mine;
    __syncthreads();
    st = s_stat[0];
    for (int w = 1; w < kLpWarps; ++w) st = stat_join(st, s_stat[w]);
    const int nkeys = kLpWarps * a.n_top;
    // the place of key i among the CTA's lists (keys are distinct but for 0, which names no score)
    auto place = [&](unsigned long long k) {
        int above = 0;
        for (int q = 0; q < nkeys; ++q) above += s_key[q] > k;
        return above;
    };
    if (a.parts > 1) {
        // the parts' results meet in scratch; the row's last CTA joins them in part order
        if constexpr (TOP) {
            unsigned long long* mine = a.part_keys + (row * a.parts + part) * a.n_top;
            for (int i = threadIdx.x; i < nkeys; i += kLpThreads) {
                const unsigned long long k = s_key[i];
                const int at = k ? place(k) : a.n_top;
                if (at < a.n_top) mine[at] = k;
            }
            const int held = __syncthreads_count(threadIdx.x < nkeys && s_key[threadIdx.x] != 0ull);
            for (int i = held + int(threadIdx.x); i < a.n_top; i += kLpThreads) mine[i] = 0ull;
        }
        if (threadIdx.x == 0) a.part_stat[row * a.parts + part] = make_float4(st.m, st.s, st.u, st.raw);
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) s_flag = atomicAdd(&a.st->row_ctr[row], 1u) == uint32_t(a.parts - 1);
        __syncthreads();
        if (!s_flag) return;
        __threadfence();
        st = stat_none();
        for (int q = 0; q < a.parts; ++q) {
            const float4 f = __ldcg(&a.part_stat[row * a.parts + q]);
            st = stat_join(st, Stat{f.x, f.y, f.z, f.w});
        }
        if (threadIdx.x == 0) a.st->row_ctr[row] = 0u;
        if constexpr (TOP) {  // each warp joins its share of the parts' lists
            l = TopList{0ull, 0ull, 0.0f};
            for (int q = warp; q < a.parts; q += kLpWarps)
                top_insert(l, lane < a.n_top ? __ldcg(a.part_keys + (row * a.parts + q) * a.n_top + lane) : 0ull, a.n_top);
            if (lane < a.n_top) s_key[warp * a.n_top + lane] = l.mine;
            __syncthreads();
        }
    }
    // P = e^((x - m) - ln_s)
    float m = st.m, ln_s, entropy;
    if (st.raw == -INFINITY) {
        m = -INFINITY;
        ln_s = entropy = 0.0f;
    } else if (!(fabsf(st.raw) <= kLpFar)) {
        m = st.raw;
        ln_s = careful_log_sum(a, DT, row, m, &entropy, s_w);
    } else {
        const float lg = log2f(st.s), resid = __fmaf_rn(m, kLpLog2e, -log2_base(m));
        ln_s = (lg - resid) * kLpLn2;
        entropy = (lg - st.u / st.s) * kLpLn2;
    }
    auto log_prob = [&](float x) { return m == -INFINITY ? -INFINITY : (x - m) - ln_s; };
    const int first = a.view_rank >= 0 ? a.view_rank : 0, last = a.view_rank >= 0 ? first + 1 : a.p;
    if (warp == 0) {
        const int tok = a.tokens[row];
        float lp = 0.0f;  // no token
        if (tok >= 0 && size_t(tok) < a.V) lp = log_prob(score_at(a, DT, row, size_t(tok)));
        else if (tok != -1 && lane == 0) raise_status(a.ctl, COLL_ERR_INVALID_ARG);
        for (int r = first + lane; r < last; r += 32) {
            a.logprob[r][row] = lp;
            if (a.entropy[r]) a.entropy[r][row] = entropy;
            if (a.lse[r]) a.lse[r][row] = m + ln_s;
        }
    }
    if constexpr (TOP) {
        for (int i = threadIdx.x; i < nkeys; i += kLpThreads) {
            const unsigned long long k = s_key[i];
            const int at = k ? place(k) : a.n_top;
            if (at >= a.n_top) continue;
            const float lp = log_prob(order_score(uint32_t(k >> 32)));
            for (int r = first; r < last; ++r) {
                a.top_idx[r][row * a.n_top + at] = int32_t(~uint32_t(k));
                a.top_logprob[r][row * a.n_top + at] = lp;
            }
        }
        // fewer scores than n are numbers: the places left name no column
        const int held = __syncthreads_count(threadIdx.x < nkeys && s_key[threadIdx.x] != 0ull);
        for (int i = held + int(threadIdx.x); i < a.n_top; i += kLpThreads)
            for (int r = first; r < last; ++r) {
                a.top_idx[r][row * a.n_top + i] = -1;
                a.top_logprob[r][row * a.n_top + i] = __int_as_float(0x7fffffff);
            }
    }
}

// ---- gradient ------------------------------------------------------------------------------------

struct RowGrad {
    float m, ln_s;  // P = e^((x - m) - ln_s): the stored lse and 0, or the row's maximum and its sum's logarithm
    float gl, ge, entropy;
};
__device__ __forceinline__ float grad_of(const RowGrad& g, float x) {
    const float lp = (x - g.m) - g.ln_s;
    const float prob = ex2(lp * kLpLog2e);
    // dx / P = -(gl + ge (ln P + H)); a score of probability 0 has no gradient, whatever its logarithm
    return prob > 0.0f ? -prob * __fmaf_rn(g.ge, lp + g.entropy, g.gl) : prob == 0.0f ? 0.0f : prob;
}

template <int DT>
__global__ void __launch_bounds__(kLpThreads) k_logprobs_grad(const __grid_constant__ LogprobArgs a) {
    using P = Pack16<DT>;
    constexpr int L = P::L, D = Elem<DT>::kBytes;
    __shared__ int s_flag;
    if (threadIdx.x == 0) s_flag = status_failed(a.ctl);
    __syncthreads();
    if (s_flag) return;
    // CTA -> (row, rank, piece of the shard's row)
    size_t b = blockIdx.x;
    const size_t piece = b % a.parts;
    b /= a.parts;
    const int r = a.view_rank >= 0 ? a.view_rank : int(b % a.p);
    const size_t row = a.view_rank >= 0 ? b : b / a.p;
    const size_t v0 = size_t(r) * a.m;                                     // first column of the shard
    const size_t all = v0 < a.V ? min(a.m, a.V - v0) : 0;                  // its columns; the rest is padding
    const char* in = static_cast<const char*>(a.logits[r]) + row * a.ld * D;
    char* out = static_cast<char*>(a.grad_logits[r]) + row * a.ld_grad * D;
    RowGrad g;
    g.m = a.lse_in[r][row];
    g.ln_s = 0.0f;
    g.ge = a.grad_entropy ? a.grad_entropy[row] : 0.0f;
    g.entropy = a.grad_entropy ? a.entropy_in[r][row] : 0.0f;
    const int tok = a.tokens[row];
    if ((tok < -1 || (tok >= 0 && size_t(tok) >= a.V)) && threadIdx.x == 0) raise_status(a.ctl, COLL_ERR_INVALID_ARG);
    g.gl = tok >= 0 ? a.grad_logprob[row] : 0.0f;
    const bool none = g.m == -INFINITY;  // a row without a distribution: zeros whatever its scores
    if (!none && !(fabsf(g.m) <= kLpFar)) {  // an fp32 lse that far out has lost the sum: take it again
        __shared__ float s_w[kLpWarps];
        float top = -INFINITY, entropy;
        for (size_t v = threadIdx.x; v < a.V; v += kLpThreads) top = max_nan(top, score_at(a, DT, row, v));
        g.m = cta_max(top, s_w);
        g.ln_s = careful_log_sum(a, DT, row, g.m, &entropy, s_w);
        g.entropy = a.grad_entropy ? entropy : 0.0f;
    }
    const size_t own = tok >= 0 && size_t(tok) >= v0 && size_t(tok) < v0 + all && !none && g.gl != 0.0f ? size_t(tok) - v0 : SIZE_MAX;
    const size_t have = none ? 0 : all;
    const size_t c0 = a.m * piece / a.parts, c1 = a.m * (piece + 1) / a.parts;
    auto value = [&](size_t c, float x) {
        float d = c < have ? grad_of(g, x) : 0.0f;
        if (c == own) d += g.gl;
        return d;
    };
    const uintptr_t ia = reinterpret_cast<uintptr_t>(in + c0 * D), oa = reinterpret_cast<uintptr_t>(out + c0 * D);
    const bool together = ((ia ^ oa) & 15) == 0;  // 16-byte boundaries fall on the same columns
    const size_t n = c1 - c0;
    const size_t head = together ? min(n, size_t((16 - (ia & 15)) & 15) / D) : n;
    const size_t vecs = together ? (n - head) / L : 0, tail = n - head - vecs * L;
    for (size_t i = threadIdx.x; i < head + tail; i += kLpThreads) {
        const size_t c = c0 + (i < head ? i : i + vecs * L);
        const float x = c < have ? load_elem<DT>(in, c) : 0.0f;
        store_elem<DT>(out, c, value(c, x));
    }
    const size_t body = c0 + head;
    for (size_t i0 = 0; i0 < vecs; i0 += kLpThreads * kLpUnroll) {
        uint4 raw[kLpUnroll];
#pragma unroll
        for (int q = 0; q < kLpUnroll; ++q) {
            const size_t i = i0 + q * kLpThreads + threadIdx.x;
            if (i < vecs) raw[q] = ld_stream_v4(in + (body + i * L) * D);
        }
#pragma unroll
        for (int q = 0; q < kLpUnroll; ++q) {
            const size_t i = i0 + q * kLpThreads + threadIdx.x;
            if (i >= vecs) break;
            const size_t c = body + i * L;
            float x[L];
            P::unpack(raw[q], x);
#pragma unroll
            for (int j = 0; j < L; ++j) x[j] = c + j < have ? grad_of(g, x[j]) : 0.0f;
            if (own - c < size_t(L)) {
#pragma unroll
                for (int j = 0; j < L; ++j)
                    if (own == c + j) x[j] += g.gl;
            }
            st_v4(out + c * D, P::pack(x));
        }
    }
}

cudaError_t launch_logprobs(const LogprobArgs& a, int dtype, cudaStream_t s) {
    const size_t ctas = a.rows * size_t(a.parts);
    if (ctas > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    auto go = [&](auto kernel) {
        kernel<<<unsigned(ctas), kLpThreads, 0, s>>>(a);
        return cudaGetLastError();
    };
    if (dtype == COLL_BF16) return a.n_top ? go(k_logprobs<COLL_BF16, true>) : go(k_logprobs<COLL_BF16, false>);
    return a.n_top ? go(k_logprobs<COLL_FP32, true>) : go(k_logprobs<COLL_FP32, false>);
}

cudaError_t launch_logprobs_grad(const LogprobArgs& args, int dtype, cudaStream_t s) {
    LogprobArgs a = args;
    constexpr size_t kPiece = 16384;  // columns of one CTA
    a.parts = int(std::max<size_t>(1, (a.m + kPiece - 1) / kPiece));
    const size_t ctas = a.rows * size_t(a.parts) * (a.view_rank >= 0 ? 1 : size_t(a.p));
    if (ctas > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    if (dtype == COLL_BF16) k_logprobs_grad<COLL_BF16><<<unsigned(ctas), kLpThreads, 0, s>>>(a);
    else k_logprobs_grad<COLL_FP32><<<unsigned(ctas), kLpThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace simcomm
