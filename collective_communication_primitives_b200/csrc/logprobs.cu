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
// by the one exponential per score. Measured on B200: 1023 x 50257 fp32 48 us, 4.3 TB/s; 2048 x 131072 bf16 105 us,
// 5.1 TB/s, with 4 alternatives 137 us (five CTAs on an SM; with four 8% and 9% more); 8 x 131072 fp32 with 8 alternatives 14.4 us.
//
// Alternatives are 64-bit keys: the score's order, then the complement of the column, so that the lower
// column wins among equals. The scan itself keeps nothing for them but each thread's maximum, which it has
// anyway: the n-th largest of the maxima of 32 groups of 8 threads is a bound that n scores reach, so only threads
// whose maximum reaches it can hold one of the n best. There are little more than n of them, ties aside, and
// their share of the columns is read again, the scores that reach the bound gathered in shared memory and sorted out. If more do than it
// holds (many equal scores), all columns are gone through again with a sorted list of the n best per warp.
//
// The exponentials are powers of two, 2^(x log2e - B) with B = M log2e rounded to fp32, so that a score
// costs one fused multiply-add and one ex2: S and U refer to B, and the rounding of B is put back at the
// end (resid below). That holds while |M| is moderate. Masked scores: -inf has probability 0; for the
// arithmetic a score below -2^40 counts as -2^40, which gives it probability 0 next to any score that is
// not masked and keeps 0 * inf out of the sums. A row whose maximum is beyond +-1e5, such as one masked
// throughout by the type's lowest value, is summed again relative to its maximum. A row of nothing but
// -inf has no distribution: lse and logprob -inf, entropy 0, gradient 0. NaN or +inf in a row makes its
// values NaN.
#include <algorithm>

#include "scores.cuh"

namespace simcomm {

constexpr int kLpGather = 768;          // keys of scores that passed the bound
constexpr float kLpFloor = -0x1p40f;    // scores below count as this in the sums (x log2e rounds alike at a power of two)
constexpr float kLpFar = 1e5f;          // rows whose maximum is further from 0 are summed again
// In the gradient, rows whose lse is further from 0 than this are summed again too: an fp32 lse is off by half its last
// place, which is the relative error of every P. 2^-18 is let pass, 2^-14 where the result is rounded to bf16.
template <int DT> constexpr float near_lse() { return DT == COLL_BF16 ? 2048.0f : 128.0f; }

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
// The join of a warp's lanes, on every lane: all relative to the largest maximum, then plain sums.
__device__ __forceinline__ Stat stat_warp(Stat a) {
    float m = a.m, raw = a.raw;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
        raw = max_nan(raw, __shfl_xor_sync(0xffffffffu, raw, d));
    }
    const float da = log2_base(a.m) - log2_base(m), fa = ex2(da);
    float s = a.s * fa, u = __fmaf_rn(s, da, a.u * fa);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, d);
        u += __shfl_xor_sync(0xffffffffu, u, d);
    }
    return Stat{m, s, u, raw};
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

// What a CTA knows of its best scores.
struct TopShared {
    uint32_t bound;   // order of a score that n of the CTA reach
    uint32_t count;   // keys gathered (more than kLpGather: some were dropped)
    uint32_t group[32];             // order of the largest number that 8 threads met, 0: none
    uint32_t threads;               // threads that reach the bound
    uint8_t thread[kLpThreads];
    unsigned long long key[kLpGather];
};

__device__ __forceinline__ void top_gather(TopShared& top, float x, uint32_t col) {
    if (x == x && score_order(x) >= top.bound) {
        const uint32_t at = atomicAdd(&top.count, 1u);
        if (at < uint32_t(kLpGather)) top.key[at] = top_key(x, col);
    }
}

// A thread's running sums, two lanes of each.
struct Feed {
    float m, raw;
    unsigned long long s, u;
};
__device__ __forceinline__ Feed feed_none() { return Feed{kLpFloor, -INFINITY, 0ull, 0ull}; }
__device__ __forceinline__ Stat feed_stat(const Feed& f) {
    float s0, s1, u0, u1;
    unpack2(f.s, s0, s1);
    unpack2(f.u, u0, u1);
    return Stat{f.m, s0 + s1, u0 + u1, f.raw};
}

// Makes the sums refer to a maximum of at least `top`.
__device__ __forceinline__ void feed_raise(Feed& f, float top) {
    if (!(top <= f.m)) {  // larger, or NaN
        const float m = top == INFINITY ? __int_as_float(0x7fffffff) : top;
        const float d = log2_base(f.m) - log2_base(m), scale = ex2(d);
        const unsigned long long dd = pack2(d, d), ss = pack2(scale, scale), zero = 0ull;
        f.s = fma2(f.s, ss, zero);
        f.u = fma2(f.s, dd, fma2(f.u, ss, zero));
        f.m = m;
    }
}

// Whether the maximum is raised for a batch of kLpUnroll vectors at once or for each as it arrives: 2-byte scores are
// bound by instructions, 4-byte ones by waiting for the loads. Measured on B200, batch and each: 106 and 109 us for 2048
// x 131072 bf16, 137 and 142 with 4 alternatives, 54 and 47 for 1023 x 50257 fp32.
template <int DT> constexpr bool by_batch() { return DT == COLL_BF16; }

// Adds one 16-byte vector of scores to a thread's sums.
template <int DT> __device__ __forceinline__ void feed_vector(Feed& f, const uint4& v) {
    constexpr int L = 16 / Elem<DT>::kBytes;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[L];
    if constexpr (!by_batch<DT>()) {
        const float top = vector_top<DT>(v);
        f.raw = max_nan(f.raw, top);
        feed_raise(f, top);
    }
    if constexpr (DT == COLL_BF16) {  // clamp on pairs
        constexpr uint32_t kFloor2 = 0xD380D380u;  // kLpFloor twice
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t c = max_nan_bf16x2(w[q], kFloor2);
            x[2 * q] = bf16_bits_to_float(c);
            x[2 * q + 1] = __uint_as_float(c & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = fmaxf(__uint_as_float(w[q]), kLpFloor);
    }
    const float base = -log2_base(f.m);
    const unsigned long long bb = pack2(base, base), ll = pack2(kLpLog2e, kLpLog2e);
#pragma unroll
    for (int q = 0; q < L; q += 2) {
        const unsigned long long d = fma2(pack2(x[q], x[q + 1]), ll, bb);
        float d0, d1;
        unpack2(d, d0, d1);
        const unsigned long long e = pack2(ex2(d0), ex2(d1));
        f.s = add2(f.s, e);
        f.u = fma2(e, d, f.u);
    }
}

// Gathers the scores that may be among the n best, given the thread's maximum (NaN: it met one). CTA-collective.
template <int DT>
__device__ __forceinline__ void gather_best(const LogprobArgs& a, size_t row, uint32_t v0, uint32_t v1, float raw, TopShared& top) {
    using P = Pack16<DT>;
    constexpr int L = P::L;
    const int lane = threadIdx.x & 31;
    // behind a NaN a thread's maximum is not known: it counts for nothing and is looked at in any case
    const uint32_t mine = raw > -INFINITY ? score_order(raw) : 0u;
    uint32_t most = mine;
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    if (threadIdx.x % 8 == 0) top.group[threadIdx.x / 8] = most;
    if (threadIdx.x == 0) top.count = top.threads = 0u;
    __syncthreads();
    // every warp finds the bound for itself: the group whose maximum has n - 1 others before it (the lower group
    // among equals); 0 where fewer than n groups have a number
    const uint32_t own = top.group[lane];
    int before = 0;
#pragma unroll
    for (int g = 0; g < 32; ++g) {
        const uint32_t other = __shfl_sync(0xffffffffu, own, g);
        before += other > own || (other == own && g < lane);
    }
    const uint32_t bound = __shfl_sync(0xffffffffu, own, __ffs(__ballot_sync(0xffffffffu, before == a.n_top - 1)) - 1);
    if (threadIdx.x == 0) top.bound = bound;
    if (raw != raw || mine >= bound) top.thread[atomicAdd(&top.threads, 1u)] = uint8_t(threadIdx.x);
    __syncthreads();
    const uint32_t nt = top.threads;
    auto offer = [&](const uint4& raw_scores, uint32_t col) {
        float x[L];
        P::unpack(raw_scores, x);
#pragma unroll
        for (int j = 0; j < L; ++j) top_gather(top, x[j], col + j);
    };
    // pieces four at a time, so that their loads are in flight together
    for (uint32_t v = v0; v < v1;) {
        uint4 got[4];
        uint32_t col[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            col[q] = 0xffffffffu;
            if (v >= v1) continue;
            const Piece<DT> pc(a, row, v, v1);
            const uint32_t turns = (pc.vecs + kLpThreads - 1) / kLpThreads;
            const int shift = turns > 1 ? 32 - __clz(turns - 1) : 0;  // turns as a power of two: no division by item
            for (uint32_t w = threadIdx.x; w < nt << shift; w += kLpThreads) {
                const uint32_t i = (w & ((1u << shift) - 1u)) * kLpThreads + top.thread[w >> shift];
                if (i >= pc.vecs) continue;
                const uint4 scores = ld_stream_v4(pc.vector(i));
                const uint32_t c = v + pc.head + i * L;
                if (w == threadIdx.x) {
                    got[q] = scores;
                    col[q] = c;
                } else {
                    offer(scores, c);
                }
            }
            if (threadIdx.x < pc.head + pc.tail) {
                const uint32_t at = pc.end_at(threadIdx.x);
                top_gather(top, load_elem<DT>(pc.base, at), v + at);
            }
            v = pc.end;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (col[q] != 0xffffffffu) offer(got[q], col[q]);
    }
    __syncthreads();
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

// The n best of the CTA's columns from a sorted list per warp, into key[0, kLpWarps * n), unsorted; the way
// that takes any number of ties. CTA-collective.
template <int DT>
__device__ __noinline__ void top_by_lists(const LogprobArgs& a, size_t row, uint32_t v0, uint32_t v1, unsigned long long* key) {
    constexpr int L = Pack16<DT>::L;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    TopList l{0ull, 0ull};
    scan_columns<DT>(a, row, v0, v1, [&](const uint4& raw, int cnt, uint32_t col) {
        float x[L];
        Pack16<DT>::unpack(raw, x);
#pragma unroll
        for (int j = 0; j < L; ++j) top_insert(l, j < cnt && x[j] == x[j] ? top_key(x[j], col + j) : 0ull, a.n_top);
    }, [](const uint4 (&)[kLpUnroll], bool) {});
    __syncthreads();
    if (lane < a.n_top) key[warp * a.n_top + lane] = l.mine;
    __syncthreads();
}

// A thread's sums over its share of the columns [v0, v1).
template <int DT> __device__ __forceinline__ Feed scan_sums(const LogprobArgs& a, size_t row, uint32_t v0, uint32_t v1) {
    Feed f = feed_none();
    // A thread's sums refer to the largest of its warp's first vectors from the start: a warp rescales where any of its
    // threads meets a larger score, and without this it did in two vectors of three (3% more for 2048 x 131072 bf16).
    auto batch = [&](const uint4 (&raw)[kLpUnroll], bool start) {
        if (!by_batch<DT>() && !start) return;
        float top = vector_top<DT>(raw[0]);
#pragma unroll
        for (int q = 1; q < kLpUnroll; ++q) top = max_nan(top, vector_top<DT>(raw[q]));
        if constexpr (by_batch<DT>()) f.raw = max_nan(f.raw, top);
        if (start)
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
        feed_raise(f, top);
    };
    scan_columns<DT>(a, row, v0, v1, [&](const uint4& raw, int, uint32_t) { feed_vector<DT>(f, raw); }, batch);
    return f;
}
// log2 of the sum of e^(x - maximum): the rounding of the sums' base is put back.
__device__ __forceinline__ float stat_log2(const Stat& st) {
    return log2f(st.s) - __fmaf_rn(st.m, kLpLog2e, -log2_base(st.m));
}

// The maximum of a row and ln of the sum of e^(x - maximum), for a moderate maximum. CTA-collective.
template <int DT> __device__ __noinline__ float2 sum_again(const LogprobArgs& a, size_t row, Stat* s_stat) {
    Stat st = stat_warp(feed_stat(scan_sums<DT>(a, row, 0, uint32_t(a.V))));
    if ((threadIdx.x & 31) == 0) s_stat[threadIdx.x >> 5] = st;
    __syncthreads();
    st = s_stat[0];
    for (int w = 1; w < kLpWarps; ++w) st = stat_join(st, s_stat[w]);
    return make_float2(st.m, stat_log2(st) * kLpLn2);
}

template <int DT, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 5) k_logprobs(const __grid_constant__ LogprobArgs a) {
    __shared__ Stat s_stat[kLpWarps];
    __shared__ TopShared s_top;
    __shared__ float s_w[kLpWarps];
    __shared__ int s_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t row = blockIdx.x / a.parts;
    const int part = int(blockIdx.x % a.parts);
    if (threadIdx.x == 0) s_flag = status_failed(a.ctl);
    __syncthreads();
    if (s_flag) return;
    const uint32_t v0 = uint32_t(a.V * part / a.parts), v1 = uint32_t(a.V * (part + 1) / a.parts);
    const Feed f = scan_sums<DT>(a, row, v0, v1);
    Stat st = stat_warp(feed_stat(f));
    if (lane == 0) s_stat[warp] = st;
    __syncthreads();
    int nkeys = 0;
    if constexpr (TOP) {
        gather_best<DT>(a, row, v0, v1, f.raw, s_top);
        nkeys = int(s_top.count);
        if (nkeys > kLpGather) {
            top_by_lists<DT>(a, row, v0, v1, s_top.key);
            nkeys = kLpWarps * a.n_top;
        }
    }
    // the place of a key among the CTA's (keys are distinct but for 0, which names no score)
    auto place = [&](unsigned long long k) {
        int above = 0;
        for (int q = 0; q < nkeys; ++q) above += s_top.key[q] > k;
        return above;
    };
    // numbers among the keys; n at most counts. Where the bound came from n scores there are as many.
    bool full = TOP && s_top.bound != 0u && nkeys <= kLpGather;
    auto held = [&]() {
        if (full) return a.n_top;
        int n = 0;
        for (int i = threadIdx.x; i < nkeys; i += kLpThreads) n += s_top.key[i] != 0ull;
        return __syncthreads_count(n > 0) >= a.n_top ? a.n_top : min(a.n_top, int(cta_sum(float(n), s_w)));
    };
    if (a.parts > 1) {
        // the parts' results meet in scratch; the row's last CTA joins them in part order
        if constexpr (TOP) {
            unsigned long long* mine = a.part_keys + (row * a.parts + part) * a.n_top;
            for (int i = threadIdx.x; i < nkeys; i += kLpThreads) {
                const unsigned long long k = s_top.key[i];
                const int at = k ? place(k) : a.n_top;
                if (at < a.n_top) mine[at] = k;
            }
            const int n = held();
            for (int i = n + int(threadIdx.x); i < a.n_top; i += kLpThreads) mine[i] = 0ull;
        }
        if (threadIdx.x == 0) {
            st = s_stat[0];
            for (int w = 1; w < kLpWarps; ++w) st = stat_join(st, s_stat[w]);
            a.part_stat[row * a.parts + part] = make_float4(st.m, st.s, st.u, st.raw);
        }
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) s_flag = atomicAdd(&a.st->row_ctr[row], 1u) == uint32_t(a.parts - 1);
        __syncthreads();
        if (!s_flag) return;
        __threadfence();
        if (threadIdx.x == 0) a.st->row_ctr[row] = 0u;
        if (warp == 0) {  // a lane's parts in order, then the lanes
            st = stat_none();
            for (int q = lane; q < a.parts; q += 32) {
                const float4 v = __ldcg(&a.part_stat[row * a.parts + q]);
                st = stat_join(st, Stat{v.x, v.y, v.z, v.w});
            }
            st = stat_warp(st);
            if (lane == 0) s_stat[0] = st;
        }
        if constexpr (TOP) {  // each warp joins its share of the parts' lists
            TopList l{0ull, 0ull};
            for (int q = warp; q < a.parts; q += kLpWarps)
                top_insert(l, lane < a.n_top ? __ldcg(a.part_keys + (row * a.parts + q) * a.n_top + lane) : 0ull, a.n_top);
            if (lane < a.n_top) s_top.key[warp * a.n_top + lane] = l.mine;
            nkeys = kLpWarps * a.n_top;
            full = false;  // of this part only
        }
        __syncthreads();
        st = s_stat[0];
    } else {
        st = s_stat[0];
        for (int w = 1; w < kLpWarps; ++w) st = stat_join(st, s_stat[w]);
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
        ln_s = stat_log2(st) * kLpLn2;
        entropy = (log2f(st.s) - st.u / st.s) * kLpLn2;
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
            const unsigned long long k = s_top.key[i];
            const int at = k ? place(k) : a.n_top;
            if (at >= a.n_top) continue;
            const float lp = log_prob(order_score(uint32_t(k >> 32)));
            for (int r = first; r < last; ++r) {
                a.top_idx[r][row * a.n_top + at] = int32_t(~uint32_t(k));
                a.top_logprob[r][row * a.n_top + at] = lp;
            }
        }
        // fewer scores than n are numbers: the places left name no column
        const int n = held();
        for (int i = n + int(threadIdx.x); i < a.n_top; i += kLpThreads)
            for (int r = first; r < last; ++r) {
                a.top_idx[r][row * a.n_top + i] = -1;
                a.top_logprob[r][row * a.n_top + i] = __int_as_float(0x7fffffff);
            }
    }
}

// ---- gradient ------------------------------------------------------------------------------------

// With d = x log2e - B, B = (m + ln_s) log2e rounded: P = 2^d c, c = 2^-(what the rounding of B left out), and
// ln P = d ln 2 + ln c. So dx = -P (gl + ge (ln P + H)) = 2^d (a0 + a1 d), two constants of the row. Bound by memory:
// 1023 x 50257 fp32 80 us, 5.1 TB/s, 2048 x 131072 bf16 207 us, 5.2 TB/s on B200 (when it was
// 79 and 202 with four CTAs on an SM, it was 78 and 221 with three, 84 and 214 with five, which spill).
struct RowGrad {
    float base, a0, a1;
};
__device__ __forceinline__ RowGrad row_grad(float m, float ln_s, float gl, float ge, float entropy) {
    RowGrad g;
    const float b_m = m * kLpLog2e, b_s = ln_s * kLpLog2e;
    g.base = b_m + b_s;
    // the sum's rounding, then the products'
    const float sum_lo = (b_m - g.base) + b_s;
    const float lo = sum_lo + __fmaf_rn(m, kLpLog2e, -b_m) + __fmaf_rn(ln_s, kLpLog2e, -b_s);
    const float c = exp2f(-lo);
    g.a0 = -c * (gl + ge * (entropy - lo * kLpLn2));
    g.a1 = -c * ge * kLpLn2;
    return g;
}
// The gradients of a vector of scores, without the given token's own term.
template <int DT> __device__ __forceinline__ uint4 grad_vector(const RowGrad& g, const uint4& v) {
    constexpr int L = Pack16<DT>::L;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[L];
    if constexpr (DT == COLL_BF16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t c = max_nan_bf16x2(w[q], 0xD380D380u);  // kLpFloor: a masked score's 2^d is 0 and d finite
            x[2 * q] = bf16_bits_to_float(c);
            x[2 * q + 1] = __uint_as_float(c & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = max_nan(__uint_as_float(w[q]), kLpFloor);
    }
    const unsigned long long ll = pack2(kLpLog2e, kLpLog2e), bb = pack2(-g.base, -g.base), a0 = pack2(g.a0, g.a0),
                             a1 = pack2(g.a1, g.a1), zero = 0ull;
#pragma unroll
    for (int q = 0; q < L; q += 2) {
        const unsigned long long d = fma2(pack2(x[q], x[q + 1]), ll, bb);
        float d0, d1;
        unpack2(d, d0, d1);
        unpack2(fma2(pack2(ex2(d0), ex2(d1)), fma2(a1, d, a0), zero), x[q], x[q + 1]);
    }
    return Pack16<DT>::pack(x);
}

template <int DT>
__global__ void __launch_bounds__(kLpThreads, 4) k_logprobs_grad(const __grid_constant__ LogprobArgs a) {
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
    float m = a.lse_in[r][row], ln_s = 0.0f;
    const float ge = a.grad_entropy ? a.grad_entropy[row] : 0.0f;
    float entropy = a.grad_entropy ? a.entropy_in[r][row] : 0.0f;
    const int tok = a.tokens[row];
    if ((tok < -1 || (tok >= 0 && size_t(tok) >= a.V)) && threadIdx.x == 0) raise_status(a.ctl, COLL_ERR_INVALID_ARG);
    const float gl = tok >= 0 ? a.grad_logprob[row] : 0.0f;
    const bool none = m == -INFINITY;  // a row without a distribution: zeros whatever its scores
    // Every CTA of a far row sums the whole row; beyond kLpFar with care. Measured on B200 with every row beyond near_lse:
    // 207 us in place of 80 for 1023 x 50257 fp32 on 4 ranks.
    if (!none && fabsf(m) > near_lse<DT>() && fabsf(m) <= kLpFar) {
        __shared__ Stat s_stat[kLpWarps];
        const float2 again = sum_again<DT>(a, row, s_stat);
        m = again.x;
        ln_s = again.y;
    } else if (!none && !(fabsf(m) <= kLpFar)) {
        __shared__ float s_w[kLpWarps];
        float top = -INFINITY, h;
        for (size_t v = threadIdx.x; v < a.V; v += kLpThreads) top = max_nan(top, score_at(a, DT, row, v));
        m = cta_max(top, s_w);
        ln_s = careful_log_sum(a, DT, row, m, &h, s_w);
        if (a.grad_entropy) entropy = h;
    }
    const bool far = !(fabsf(m) <= kLpFar);  // the scores' differences from m need more than a fused product
    const RowGrad g = row_grad(m, ln_s, gl, ge, entropy);
    const size_t own = tok >= 0 && size_t(tok) >= v0 && size_t(tok) < v0 + all && !none && gl != 0.0f ? size_t(tok) - v0 : SIZE_MAX;
    const size_t have = none ? 0 : all;
    const size_t c0 = a.m * piece / a.parts, c1 = a.m * (piece + 1) / a.parts;
    auto value = [&](size_t c) {  // one column's gradient
        if (c >= have) return 0.0f;
        const float x = load_elem<DT>(in, c), lp = (x - m) - ln_s, prob = ex2(lp * kLpLog2e);
        const float d = prob > 0.0f ? -prob * __fmaf_rn(ge, lp + entropy, gl) : prob == 0.0f ? 0.0f : prob;
        return c == own ? d + gl : d;
    };
    const uintptr_t ia = reinterpret_cast<uintptr_t>(in + c0 * D), oa = reinterpret_cast<uintptr_t>(out + c0 * D);
    const bool together = ((ia ^ oa) & 15) == 0 && !far;  // 16-byte boundaries fall on the same columns
    const size_t n = c1 - c0;
    const size_t head = together ? min(n, size_t((16 - (ia & 15)) & 15) / D) : n;
    // whole vectors of the shard's own columns; what is left of them and the padding go one by one
    const size_t vecs = together && have > c0 + head ? (min(c1, have) - c0 - head) / L : 0, rest = n - head - vecs * L;
    for (size_t i = threadIdx.x; i < head + rest; i += kLpThreads) {
        const size_t c = c0 + (i < head ? i : i + vecs * L);
        store_elem<DT>(out, c, value(c));
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
            st_v4(out + c * D, grad_vector<DT>(g, raw[q]));
            if (own - c < size_t(L)) store_elem<DT>(out, own, value(own));
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
    // Columns of one CTA. Measured on B200 with 4096, 16384 and 65536: 109, 79, 79 us for 1023 x 50257 fp32 on 4 ranks,
    // 371, 202, 202 for 2048 x 131072 bf16 on 8, 6.2, 6.2, 10.4 for 8 x 50257 bf16 on one.
    constexpr size_t kPiece = 16384;
    a.parts = int(std::max<size_t>(1, (a.m + kPiece - 1) / kPiece));
    const size_t ctas = a.rows * size_t(a.parts) * (a.view_rank >= 0 ? 1 : size_t(a.p));
    if (ctas > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    if (dtype == COLL_BF16) k_logprobs_grad<COLL_BF16><<<unsigned(ctas), kLpThreads, 0, s>>>(a);
    else k_logprobs_grad<COLL_FP32><<<unsigned(ctas), kLpThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace simcomm
