// Loss against a teacher's best columns, over a vocabulary whose columns are sharded over the ranks, and the gradient
// of the scores.
//
//   P = softmax(x / T) over all V columns; q over the teacher's n places: softmax(value / T), or e^value with one more
//   class for the columns that are not listed, Q = 1 - sum q and P_rest = sum of their P
//   loss = sum q (ln q - ln P) + Q (ln Q - ln P_rest)
//   dx[v] = g / T (A P[v] - q[v]),  A = sum q + Q;  off the list, with the class of the rest, g / T P[v] (A - Q / P_rest)
//
// Forward: one pass over the scores with a running maximum and sum, as in the log probabilities; few rows are cut into
// parts that the last CTA joins in order, and the last CTA of a row does the list. With the class of the rest the
// pass leaves the listed columns out, so that P_rest is a sum and no difference: what is left beside a peaked
// distribution keeps its precision. Two words of a thread, a bit for each of its vectors modulo 64, tell which have a listed
// column, a table of them which of their scores are listed.
//
// Differences x - m are formed before they are scaled, so the sums are as exact for scores far from 0 as for others, and
// a row of the type's lowest value is a row like any other. A row of nothing but -inf has P = 0.
//
// Gradient: off the list dx = 2^((x - m) c) g / T k with two constants of the row, k = A / s of the row's maximum m and sum s;
// with the class of the rest m and s are those of the rest and k = (A P_rest - Q) / s, which stays finite where P_rest
// vanishes. s is at least 1 and at most V, so that k neither overflows nor vanishes, and it is formed in 64 bits: with the logarithm of s,
// subtracted from the exponent in 32, the results were off by up to 2^-20. Then the CTA writes the listed columns
// among its own over it. Both are bound by the scores' bytes, the forward pass for 2-byte scores by instructions: one exponential
// each and its sum. Measured on B200, us forward and gradient: 2048 x 131072 bf16, 32 places and the rest, 118 and 186 (537 MB,
// 4.5 TB/s, and 1074 MB, 5.8; with a filter looked up for every vector the forward pass took 125, 75% of the issue slots
// used); 1023 x 50257 fp32, 20 places, 48 and 65 (4.3 and 6.3); 16 x 131072 fp32, 11 and 9.
#include <algorithm>
#include <cfloat>

#include "scores.cuh"

namespace simcomm {

constexpr uint32_t kFilterBatches = 16;   // a bit per vector of so many of a thread's batches
constexpr int kTable = 512;               // at least twice the places
constexpr uint32_t kEmpty = 0xffffffffu;  // no column: a vocabulary has fewer than 2^31

// Sum s of 2^((x - m) c) over a set of scores with maximum m (at least -FLT_MAX; NaN if a score is).
struct Mass {
    float m, s;
};
__device__ __forceinline__ Mass mass_none() { return Mass{-FLT_MAX, 0.0f}; }
__device__ __forceinline__ float mass_at(const Mass& a, float m, float c) { return a.s * ex2((a.m - m) * c); }
__device__ __forceinline__ Mass mass_join(const Mass& a, const Mass& b, float c) {
    const float m = max_nan(a.m, b.m);
    return Mass{m, mass_at(a, m, c) + mass_at(b, m, c)};
}
__device__ __forceinline__ Mass mass_warp(const Mass& a, float c) {
    float m = a.m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    float s = mass_at(a, m, c);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return Mass{m, s};
}

// The listed columns of a row, and where they lie in its vectors.
struct Listed {
    int32_t id[kDistillMaxTop];
    uint32_t filter[kFilterBatches / 8][kLpThreads];
    uint32_t key[kTable];    // first column of a vector with listed columns
    uint32_t mask[kTable];   // which of its columns are
};
// Batches of vectors: a CTA's threads take kLpUnroll vectors each at a time. The first of a shard has this number, modulo
// kFilterBatches, whose vectors have four bits of a thread's words.
static_assert(kLpUnroll == 4, "eight batches to a word");
template <int DT> __device__ __forceinline__ uint32_t first_batch(const DistillArgs& a, uint32_t rank) {
    return rank * (uint32_t(a.m) / (Pack16<DT>::L * kLpThreads * kLpUnroll) + 1);
}
// A column's first place among the table's.
__device__ __forceinline__ uint32_t table_at(uint32_t col) { return (col * 2654435761u) >> 23; }
static_assert(kTable == 512, "table_at gives 9 bits");

// Which of a vector's columns are listed.
__device__ __forceinline__ uint32_t listed_in(const Listed& s, uint32_t col) {
    for (uint32_t at = table_at(col), k = 0; k < kTable; at = (at + 1) % kTable, ++k) {
        if (s.key[at] == col) return s.mask[at];
        if (s.key[at] == kEmpty) break;
    }
    return 0u;
}
template <int DT> __device__ __forceinline__ void leave_out(uint4& v, uint32_t mask) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int l = 0; l < Pack16<DT>::L; ++l)
        if ((mask >> l) & 1u) {
            if constexpr (DT == COLL_BF16)
                w[l / 2] = l % 2 ? (w[l / 2] & 0xffffu) | 0xff800000u : (w[l / 2] & 0xffff0000u) | 0xff80u;
            else
                w[l] = 0xff800000u;
        }
    v = make_uint4(w[0], w[1], w[2], w[3]);
}

// The place of a column in the table, which is put there if it is not there yet.
__device__ __forceinline__ uint32_t enter(Listed& s, uint32_t col, bool* there = nullptr) {
    uint32_t at = table_at(col);
    while (true) {  // ends: the table has more places than there are columns
        const uint32_t was = atomicCAS(&s.key[at], kEmpty, col);
        if (was == kEmpty || was == col) {
            if (there) *there = was == col;
            return at;
        }
        at = (at + 1) % kTable;
    }
}

// Enters the listed columns among [v0, v1). CTA-collective; id is set.
template <int DT> __device__ __forceinline__ void list_columns(const DistillArgs& a, size_t row, uint32_t v0, uint32_t v1, Listed& s) {
#pragma unroll
    for (uint32_t i = 0; i < kFilterBatches / 8; ++i) s.filter[i][threadIdx.x] = 0u;
    for (int i = threadIdx.x; i < kTable; i += kLpThreads) {
        s.key[i] = kEmpty;
        s.mask[i] = 0u;
    }
    __syncthreads();
    const uint32_t id = int(threadIdx.x) < a.n ? uint32_t(s.id[threadIdx.x]) : kEmpty;
    if (id >= v0 && id < v1) {
        const uint32_t m = uint32_t(a.m), first = max(v0, id / m * m);
        const Piece<DT> pc(a, row, first, v1);
        const uint32_t k = id - first;
        constexpr int L = Piece<DT>::L;
        // a score outside of the whole vectors stands for itself
        const bool vector = k >= pc.head && k < pc.head + pc.vecs * L;
        const uint32_t l = vector ? (k - pc.head) % L : 0u, col = id - l;
        if (vector) {
            const uint32_t i = (k - pc.head) / L, batch = first_batch<DT>(a, id / m) + i / (kLpThreads * kLpUnroll);
            atomicOr(&s.filter[batch / 8 % (kFilterBatches / 8)][i % kLpThreads], 1u << (batch % 8 * 4 + i / kLpThreads % kLpUnroll));
        }
        atomicOr(&s.mask[enter(s, col)], 1u << l);
    }
    __syncthreads();
}

// A thread's next vectors of a piece, from vector i0 on; missing ones are -inf.
template <int DT> __device__ __forceinline__ void load_batch(const Piece<DT>& pc, uint32_t i0, uint4 (&raw)[kLpUnroll]) {
    constexpr uint32_t kNone = DT == COLL_BF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
#pragma unroll
    for (int q = 0; q < kLpUnroll; ++q) {
        const uint32_t i = i0 + q * kLpThreads + threadIdx.x;
        raw[q] = i < pc.vecs ? ld_stream_v4(pc.vector(i)) : make_uint4(kNone, kNone, kNone, kNone);
    }
}

// A thread's sum over its share of the columns [v0, v1), without the listed ones if REST. raw: the first piece's first vectors.
template <int DT, bool REST>
__device__ __forceinline__ Mass sum_columns(const DistillArgs& a, size_t row, uint32_t v0, uint32_t v1, float c, const Listed& list,
                                            uint4 (&raw)[kLpUnroll]) {
    constexpr int L = Pack16<DT>::L;
    float m = -FLT_MAX;
    unsigned long long s = 0ull;
    const unsigned long long cc = pack2(c, c), zero = 0ull;
    static_assert(kFilterBatches == 16, "two words");
    const uint32_t filter0 = REST ? list.filter[0][threadIdx.x] : 0u, filter1 = REST ? list.filter[1][threadIdx.x] : 0u;
    auto raise = [&](float top) {
        if (!(top <= m)) {  // larger, or NaN
            const float f = ex2((m - top) * c);
            s = fma2(s, pack2(f, f), zero);
            m = top;
        }
    };
    auto add = [&](const uint4& v) {
        float x[L];
        Pack16<DT>::unpack(v, x);
        const unsigned long long mm = pack2(-m, -m);
#pragma unroll
        for (int q = 0; q < L; q += 2) {
            float d0, d1;
            unpack2(mul2(add2(pack2(x[q], x[q + 1]), mm), cc), d0, d1);
            s = add2(s, pack2(ex2(d0), ex2(d1)));
        }
    };
    for (uint32_t v = v0; v < v1;) {
        const Piece<DT> pc(a, row, v, v1);
        if (threadIdx.x < pc.head + pc.tail) {  // scores before and behind the whole vectors
            const uint32_t at = pc.end_at(threadIdx.x);
            float x = load_elem<DT>(pc.base, at);
            if constexpr (REST)
                if (listed_in(list, v + at)) x = -INFINITY;
            raise(x);
            s = add2(s, pack2(ex2((x - m) * c), 0.0f));
        }
        uint32_t batch = REST ? first_batch<DT>(a, v / uint32_t(a.m)) : 0u;
        for (uint32_t i0 = 0; i0 < pc.vecs; i0 += kLpThreads * kLpUnroll, ++batch) {
            if (i0 > 0 || v != v0) load_batch<DT>(pc, i0, raw);
            if constexpr (REST) {
                const uint32_t hit = ((batch & 8 ? filter1 : filter0) >> (batch % 8 * 4)) & 15u;
                if (hit) {
#pragma unroll
                    for (int q = 0; q < kLpUnroll; ++q)
                        if ((hit >> q) & 1u) leave_out<DT>(raw[q], listed_in(list, v + pc.head + (i0 + q * kLpThreads + threadIdx.x) * L));
                }
            }
            float top = vector_top<DT>(raw[0]);
#pragma unroll
            for (int q = 1; q < kLpUnroll; ++q) top = max_nan(top, vector_top<DT>(raw[q]));
            raise(top);
#pragma unroll
            for (int q = 0; q < kLpUnroll; ++q) {
                if (i0 + q * kLpThreads + (threadIdx.x & ~31u) >= pc.vecs) break;  // none of this warp's
                add(raw[q]);
            }
        }
        v = pc.end;
    }
    float s0, s1;
    unpack2(s, s0, s1);
    return Mass{m, s0 + s1};
}

// CTAs on an SM, measured on B200, forward and gradient together, us: 2048 x 131072 bf16 with 5 and 6 310, with 4 and 5 316, with
// 5 and 4 329; 1023 x 50257 fp32 with 4 and 6 116, with 5 and 5 121, with 5 and 4 125, with 6 and 5 127.
template <int DT, bool TAIL> __global__ void __launch_bounds__(kLpThreads, DT == COLL_BF16 ? 5 : 4) k_distill(const __grid_constant__ DistillArgs a) {
    __shared__ Listed s_list;
    __shared__ Mass s_mass[kLpWarps];
    __shared__ float s_w[kLpWarps];
    __shared__ double s_d[kLpWarps];
    __shared__ int s_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = threadIdx.x;
    const size_t row = blockIdx.x / a.parts;
    const int part = int(blockIdx.x % a.parts);
    const float c = a.log2e_over;
    const uint32_t v0 = uint32_t(a.V * part / a.parts), v1 = uint32_t(a.V * (part + 1) / a.parts);
    uint4 raw[kLpUnroll];  // on their way while the list is put together
    load_batch<DT>(Piece<DT>(a, row, v0, v1), 0, raw);
    if (t == 0) s_flag = status_failed(a.ctl);
    int32_t id = -1;  // of the thread's place
    if (t < a.n) {
        id = a.top_idx[row * a.n + t];
        if (id < -1 || (id >= 0 && size_t(id) >= a.V)) {
            raise_status(a.ctl, COLL_ERR_INVALID_ARG);
            id = -1;
        }
        s_list.id[t] = id;
    }
    __syncthreads();
    if (s_flag) return;
    if constexpr (TAIL) list_columns<DT>(a, row, v0, v1, s_list);
    // a place's score and value, needed at the end only; with parts, where the last CTA alone needs them, read there
    const bool given = id >= 0;
    float x = -INFINITY, value = -INFINITY;
    auto read_place = [&]() {
        if (!given) return;
        x = score_at(a, DT, row, size_t(id));
        value = a.top_value[row * a.n + t];
    };
    if (a.parts == 1) read_place();
    Mass all = mass_warp(sum_columns<DT, TAIL>(a, row, v0, v1, c, s_list, raw), c);
    if (lane == 0) s_mass[warp] = all;
    __syncthreads();
    all = s_mass[0];
    for (int w = 1; w < kLpWarps; ++w) all = mass_join(all, s_mass[w], c);
    if (a.parts > 1) {
        // the parts' sums meet in scratch; the row's last CTA joins them in part order
        if (t == 0) {
            a.part_stat[row * a.parts + part] = make_float2(all.m, all.s);
            __threadfence();
            s_flag = atomicAdd(&a.st->row_ctr[row], 1u) == uint32_t(a.parts - 1);
        }
        __syncthreads();
        if (!s_flag) return;
        __threadfence();
        read_place();
        if (t == 0) a.st->row_ctr[row] = 0u;
        if (warp == 0) {
            all = mass_none();
            for (int q = lane; q < a.parts; q += 32) {
                const float2 v = __ldcg(&a.part_stat[row * a.parts + q]);
                all = mass_join(all, Mass{v.x, v.y}, c);
            }
            all = mass_warp(all, c);
            if (lane == 0) s_mass[0] = all;
        }
        __syncthreads();
        all = s_mass[0];
    }
    const Mass rest = all;  // with TAIL of the columns that are not listed
    // The loss is a small difference of terms of the size of ln V: they are formed and added in 64 bits (in 32 the losses of 16
    // rows of 131072 were off by 3e-6 of their size), a few operations to a place. The listed columns' part of the sum too: with
    // it the error of the rest's sum, 1e-7 of it, enters the loss times the difference of P_rest and Q only.
    const double inv_t = a.inv_temperature;
    double total = all.s;
    if constexpr (TAIL) {
        // a column's first place counts. Whether any column has two is seen in a table of all of them
        for (int i = t; i < kTable; i += kLpThreads) s_list.key[i] = kEmpty;
        __syncthreads();
        bool first = given, twice = false;
        if (given) enter(s_list, uint32_t(id), &twice);
        if (__syncthreads_or(twice))
            for (int j = 0; j < t && j < a.n && first; ++j) first = s_list.id[j] != id;
        all.m = max_nan(rest.m, cta_max(first ? max_nan(x, -FLT_MAX) : -FLT_MAX, s_w));
        total = double(rest.s) * exp((double(rest.m) - double(all.m)) * inv_t) +
                cta_sum(first ? exp((double(x) - double(all.m)) * inv_t) : 0.0, s_d);
    }
    const bool none = total == 0.0;  // nothing but -inf
    const double ln_s = none ? 0.0 : log(total);
    const double lp = none ? -double(INFINITY) : (double(x) - double(all.m)) * inv_t - ln_s;
    float top = 0.0f;
    double inv_z = 1.0, q, lq;
    if constexpr (TAIL) {
        lq = value;
        q = exp(lq);
    } else {
        top = cta_max(value, s_w);
        if (top == -INFINITY) top = 0.0f;  // no teacher
        lq = (double(value) - double(top)) * inv_t;
        q = exp(lq);
        const double z = cta_sum(q, s_d);
        inv_z = z == 0.0 ? 0.0 : 1.0 / z;
        q *= inv_z;
        lq -= log(z);
    }
    double weight = cta_sum(q, s_d), loss = cta_sum(q > 0.0 ? q * (lq - lp) : q, s_d), k = weight;
    if constexpr (TAIL) {
        double left = 1.0 - weight;
        if (left < 0x1p-20) left = 0.0;
        const double ln_rest = rest.s == 0.0f ? -double(INFINITY) : ((double(rest.m) - double(all.m)) * inv_t + log(double(rest.s))) - ln_s;
        if (left != 0.0) loss += left * (log(left) - ln_rest);
        weight += left;
        k = weight * exp(ln_rest) - left;
    }
    const int first = a.view_rank >= 0 ? a.view_rank : 0, last = a.view_rank >= 0 ? first + 1 : a.p;
    for (int r = first + t; r < last; r += kLpThreads) {
        a.loss[r][row] = float(loss);
        if (!a.stats[r]) continue;
        const bool empty = rest.s == 0.0f;  // no column off the list has a probability
        float* o = a.stats[r] + row * kDistillStats;
        o[0] = empty ? 0.0f : rest.m;
        o[1] = empty ? 0.0f : float(k / double(rest.s));
        o[2] = none ? 0.0f : all.m;
        o[3] = none ? 0.0f : float(weight / total);  // 0: no teacher, or nothing but -inf
        o[4] = top;
        o[5] = none ? 0.0f : float(inv_z);
        o[6] = o[7] = 0.0f;
    }
}

// ---- gradient ------------------------------------------------------------------------------------

// Sums a row's gradient refers to.
struct RowSlope {
    float m, k;
};
template <int DT> __device__ __forceinline__ uint4 slope_vector(const RowSlope& g, float c, const uint4& v) {
    constexpr int L = Pack16<DT>::L;
    float x[L];
    Pack16<DT>::unpack(v, x);
    const unsigned long long mm = pack2(-g.m, -g.m), cc = pack2(c, c), kk = pack2(g.k, g.k);
#pragma unroll
    for (int q = 0; q < L; q += 2) {
        float d0, d1;
        unpack2(mul2(add2(pack2(x[q], x[q + 1]), mm), cc), d0, d1);
        unpack2(mul2(pack2(ex2(d0), ex2(d1)), kk), x[q], x[q + 1]);
    }
    return Pack16<DT>::pack(x);
}

template <int DT> __global__ void __launch_bounds__(kLpThreads, 6) k_distill_grad(const __grid_constant__ DistillArgs a) {
    constexpr int L = Pack16<DT>::L, D = Elem<DT>::kBytes;
    __shared__ int32_t s_id[kDistillMaxTop];
    __shared__ float s_q[kDistillMaxTop];
    __shared__ uint32_t s_key[kTable], s_first[kTable];  // columns of this piece that are listed, and their first places
    __shared__ int s_flag;
    const int t = threadIdx.x;
    for (int i = t; i < kTable; i += kLpThreads) s_key[i] = s_first[i] = kEmpty;
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
    const size_t c0 = a.m * piece / a.parts, c1 = a.m * (piece + 1) / a.parts, n = c1 - c0;
    const uintptr_t ia = reinterpret_cast<uintptr_t>(in + c0 * D), oa = reinterpret_cast<uintptr_t>(out + c0 * D);
    const bool together = ((ia ^ oa) & 15) == 0;  // 16-byte boundaries fall on the same columns
    const size_t head = together ? min(n, size_t((16 - (ia & 15)) & 15) / D) : n, body = c0 + head;
    // whole vectors of the shard's own columns; what is left of them and the padding go one by one
    size_t vecs = together && all > body ? (min(c1, all) - body) / L : 0;
    uint4 raw[kLpUnroll];
    auto fetch = [&](size_t i0) {
#pragma unroll
        for (int q = 0; q < kLpUnroll; ++q) {
            const size_t i = i0 + q * kLpThreads + t;
            if (i < vecs) raw[q] = ld_stream_v4(in + (body + i * L) * D);
        }
    };
    fetch(0);  // on their way while the row's numbers are read
    const float* st = a.stats_in[r] + row * kDistillStats;
    if (t == 0) s_flag = status_failed(a.ctl);
    const float c = a.log2e_over, g = float(a.grad_loss[row] * a.inv_temperature), scale = st[3];
    const RowSlope slope{st[0], st[1] * g};
    int32_t id = -1;
    if (t < a.n) {
        id = a.top_idx[row * a.n + t];
        if (id < -1 || (id >= 0 && size_t(id) >= a.V)) {
            raise_status(a.ctl, COLL_ERR_INVALID_ARG);
            id = -1;
        }
        s_id[t] = id;
        s_q[t] = id < 0 ? 0.0f : expf(float((a.top_value[row * a.n + t] - st[4]) * a.inv_temperature)) * st[5];
    }
    __syncthreads();
    if (s_flag) return;
    const bool zero = scale == 0.0f;  // no teacher, or nothing but -inf
    const size_t have = zero ? 0 : all;
    if (zero) vecs = 0;
    const size_t rest = n - head - vecs * L;
    // the thread's place, if its column is one of this piece and it is the column's first: written at the end, over what the
    // pass writes there
    const size_t at = size_t(uint32_t(id)) - v0;
    bool mine = !zero && id >= 0 && size_t(id) >= v0 && at >= c0 && at < min(c1, all);
    float mine_q = 0.0f, mine_x = 0.0f;
    uint32_t place = 0;
    bool twice = false;
    if (mine) {
        mine_x = load_elem<DT>(in, at);
        mine_q = s_q[t];
        place = table_at(uint32_t(id));
        while (true) {  // ends: the table has more places than there are columns
            const uint32_t was = atomicCAS(&s_key[place], kEmpty, uint32_t(id));
            twice = was == uint32_t(id);
            if (was == kEmpty || twice) break;
            place = (place + 1) % kTable;
        }
        atomicMin(&s_first[place], uint32_t(t));
    }
    // (a comparison of every place with every other took 296 us of 478 with 256 places, 2048 x 131072 bf16 on 8 ranks)
    if (__syncthreads_or(twice) && mine) {
        mine = s_first[place] == uint32_t(t);
        mine_q = 0.0f;
        for (int j = 0; mine && j < a.n; ++j)
            if (s_id[j] == id) mine_q += s_q[j];
    }
    for (size_t i = t; i < head + rest; i += kLpThreads) {
        const size_t at = c0 + (i < head ? i : i + vecs * L);
        float y = 0.0f;
        if (at < have) y = ex2((load_elem<DT>(in, at) - slope.m) * c) * slope.k;
        store_elem<DT>(out, at, y);
    }
    for (size_t i0 = 0; i0 < vecs; i0 += kLpThreads * kLpUnroll) {
        if (i0 > 0) fetch(i0);
#pragma unroll
        for (int q = 0; q < kLpUnroll; ++q) {
            const size_t i = i0 + q * kLpThreads + t;
            if (i >= vecs) break;
            st_v4(out + (body + i * L) * D, slope_vector<DT>(slope, c, raw[q]));
        }
    }
    __syncthreads();
    if (!mine) return;
    const float p = expf(float((mine_x - st[2]) * a.inv_temperature)) * scale;  // A P
    store_elem<DT>(out, at, g * (p - mine_q));
}

cudaError_t launch_distill(const DistillArgs& a, int dtype, cudaStream_t s) {
    const size_t ctas = a.rows * size_t(a.parts);
    if (ctas > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    auto go = [&](auto kernel) {
        kernel<<<unsigned(ctas), kLpThreads, 0, s>>>(a);
        return cudaGetLastError();
    };
    if (dtype == COLL_BF16) return a.tail ? go(k_distill<COLL_BF16, true>) : go(k_distill<COLL_BF16, false>);
    return a.tail ? go(k_distill<COLL_FP32, true>) : go(k_distill<COLL_FP32, false>);
}

cudaError_t launch_distill_grad(const DistillArgs& args, int dtype, cudaStream_t s) {
    DistillArgs a = args;
    constexpr size_t kPiece = 16384;  // columns of one CTA, as in the gradient of the log probabilities
    a.parts = int(std::max<size_t>(1, (a.m + kPiece - 1) / kPiece));
    const size_t ctas = a.rows * size_t(a.parts) * (a.view_rank >= 0 ? 1 : size_t(a.p));
    if (ctas > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    if (dtype == COLL_BF16) k_distill_grad<COLL_BF16><<<unsigned(ctas), kLpThreads, 0, s>>>(a);
    else k_distill_grad<COLL_FP32><<<unsigned(ctas), kLpThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace simcomm
