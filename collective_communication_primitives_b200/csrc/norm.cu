// Root-mean-square norm of rows that lie on the ranks as partial sums, with the AllReduce before it, the residual's
// addition and 8-bit rows; and its gradient.
//
//   h = sum_q x[q] + residual,  y = h w r,  r = 1 / sqrt(mean h^2 + eps);  8 bits: scale = max |y| / 448 per group, q = y / scale
//   gradient, g = sum_q grad_out[q]:  u = h r,  dh = r (w g - u mean(w g u)) + grad_total,  dw = sum over rows of g u
//
// One CTA has a row. Its threads keep the sum of all ranks' partial rows in registers, so that every input is read once,
// and write the finished row to every rank: p + 1 rows in, p (2 bytes or more) rows out. Bound by these bytes; for a few
// rows by the latency of one load, one reduction and one store. Rows too long for registers are summed again for
// each use. Measured on B200, 8 ranks bf16, replayed in a graph: 1 row of 4096 4.7 us; 2048 rows of 4096 with total and 8-bit
// rows in groups of 128 66.5 us (355 MB: 5.3 TB/s; a row written to 8 ranks by bulk stores alone reaches 5.9), total and norm 72 us and
// their gradient 59.5 and 6 us (721 MB in 141 us: 5.1). Arithmetic takes two elements at a time: with one the gradient took 65.
//
// In the gradient a CTA takes every ctas-th row and keeps its sums of the weight's gradient in registers; a second kernel
// adds the CTAs' sums in order.
//
// Squares of |h| beyond 2^52 or so may pass fp32: such a row is summed again scaled by 2^-80 (2^24 squares of 2^48 do not),
// next to which eps is nothing.
#include <cuda_fp8.h>

#include <algorithm>
#include <cfloat>

#include "common.cuh"

namespace simcomm {

constexpr float kNormDown = 0x1p-80f;    // the scale of rows whose squares pass fp32

// Units of L elements: 16-byte vectors, or single elements where rows are not whole vectors.
template <int DT, int L> struct Unit {
    static constexpr int D = Elem<DT>::kBytes;
    using Raw = uint4;
    __device__ static Raw load(const void* base, size_t e) { return ld_stream_v4(static_cast<const char*>(base) + e * D); }
    __device__ static void unpack(const Raw& v, float (&a)[L]) { Pack16<DT>::unpack(v, a); }
    __device__ static Raw pack(const float (&a)[L]) { return Pack16<DT>::pack(a); }
    __device__ static void store(void* base, size_t e, const Raw& v) { st_v4(static_cast<char*>(base) + e * D, v); }
};
template <int DT> struct Unit<DT, 1> {
    using Raw = float;
    __device__ static Raw load(const void* base, size_t e) { return load_elem<DT>(base, e); }
    __device__ static void unpack(const Raw& v, float (&a)[1]) { a[0] = v; }
    __device__ static Raw pack(const float (&a)[1]) { return a[0]; }
    __device__ static void store(void* base, size_t e, const Raw& v) { store_elem<DT>(base, e, v); }
};
// A unit to the same place of every rank's buffer.
template <int DT, int L> __device__ __forceinline__ void store_all(const NormArgs& a, void* const (&to)[kMaxRanks], size_t e, const float (&v)[L]) {
    const typename Unit<DT, L>::Raw raw = Unit<DT, L>::pack(v);
#pragma unroll 4
    for (int r = a.rank0; r < a.rank0 + a.ranks; ++r) Unit<DT, L>::store(to[r], e, raw);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
// The n threads that compute (whole warps, from thread 0 on) meet; whether any of them is `bad`.
__device__ __forceinline__ bool meet(int n, bool bad) {
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(any) : "r"(uint32_t(bad)), "r"(n) : "memory");
    return any != 0u;
}
// Their sums of two values each, in a fixed order, the same for every thread. Rows that follow each other use two
// buffers in turn: what a thread writes for one row the others have read two rows ago, before they met for the last one.
__device__ __forceinline__ float2 cta_sum2(float a, float b, float2 (&buf)[32], int n, bool& bad) {
    const int lane = threadIdx.x & 31;
    a = warp_sum(a);
    b = warp_sum(b);
    if (lane == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
    bad = meet(n, bad);
    const float2 v = lane < n >> 5 ? buf[lane] : make_float2(0.0f, 0.0f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// |v| as a whole number in the values' order, NaN above all.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale of a group from its largest |y|, and y / scale (0 where all are 0). With the rounded reciprocal in place of the
// division a y near the middle between two 8-bit values goes to the wrong one more often: the error of the 8-bit rows of
// 2048 x 4096 bf16 was over 1.5 times that of the division, and the time the same.
__device__ __forceinline__ float scale_of(float most) {
    return most > 0.0f ? fmaxf(most / 448.0f, FLT_MIN) : most;  // 0 and NaN stay
}
__device__ __forceinline__ float over(float y, float scale) { return scale == 0.0f ? 0.0f : y / scale; }
__device__ __forceinline__ uint8_t e4m3(float v) {
    return uint8_t(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}
template <int L> struct Q8 {
    using T = uint8_t;
    __device__ static T pack(const float (&v)[1]) { return e4m3(v[0]); }
};
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
template <> struct Q8<4> {
    using T = uint32_t;
    __device__ static T pack(const float (&v)[4]) { return e4m3x4(v[0], v[1], v[2], v[3]); }
};
template <> struct Q8<8> {
    using T = uint2;
    __device__ static T pack(const float (&v)[8]) {
        return make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
    }
};

// Units' elements two at a time.
template <int L> __device__ __forceinline__ void add_to(float (&h)[L], const float (&x)[L]) {
    if constexpr (L % 2 == 0) {
#pragma unroll
        for (int l = 0; l < L; l += 2) unpack2(add2(pack2(h[l], h[l + 1]), pack2(x[l], x[l + 1])), h[l], h[l + 1]);
    } else {
#pragma unroll
        for (int l = 0; l < L; ++l) h[l] += x[l];
    }
}
// a = a b, with b a factor per element or one for all
template <int L> __device__ __forceinline__ void mul_by(float (&a)[L], const float (&b)[L]) {
    if constexpr (L % 2 == 0) {
#pragma unroll
        for (int l = 0; l < L; l += 2) unpack2(mul2(pack2(a[l], a[l + 1]), pack2(b[l], b[l + 1])), a[l], a[l + 1]);
    } else {
#pragma unroll
        for (int l = 0; l < L; ++l) a[l] *= b[l];
    }
}
template <int L> __device__ __forceinline__ void mul_by(float (&a)[L], float b) {
    float f[L];
#pragma unroll
    for (int l = 0; l < L; ++l) f[l] = b;
    mul_by<L>(a, f);
}
// c = a b + c
template <int L> __device__ __forceinline__ void mul_add(const float (&a)[L], const float (&b)[L], float (&c)[L]) {
    if constexpr (L % 2 == 0) {
#pragma unroll
        for (int l = 0; l < L; l += 2)
            unpack2(fma2(pack2(a[l], a[l + 1]), pack2(b[l], b[l + 1]), pack2(c[l], c[l + 1])), c[l], c[l + 1]);
    } else {
#pragma unroll
        for (int l = 0; l < L; ++l) c[l] = fmaf(a[l], b[l], c[l]);
    }
}
// The sum of a b over all units: an even and an odd chain
template <int L, int V> __device__ __forceinline__ float dot(const float (&a)[V][L], const float (&b)[V][L]) {
    if constexpr (L % 2 == 0) {
        unsigned long long s = 0ull;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int l = 0; l < L; l += 2) s = fma2(pack2(a[v][l], a[v][l + 1]), pack2(b[v][l], b[v][l + 1]), s);
        float even, odd;
        unpack2(s, even, odd);
        return even + odd;
    } else {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int l = 0; l < L; ++l) s = fmaf(a[v][l], b[v][l], s);
        return s;
    }
}

// The sum of all ranks' units, V of them per thread (unit v at element e0 + (v blockDim + tid) L), loads of as many ranks
// in flight as registers allow.
template <int DT, int L, int V>
__device__ __forceinline__ void sum_ranks(const NormArgs& a, size_t row, float (&h)[V][L]) {
    using U = Unit<DT, L>;
    constexpr int kAhead = V >= 8 ? 1 : 8 / V;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int l = 0; l < L; ++l) h[v][l] = -0.0f;  // the first addition leaves what it adds
    for (int q0 = 0; q0 < a.p; q0 += kAhead) {
        typename U::Raw raw[kAhead][V];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t e = (v * blockDim.x + threadIdx.x) * L;
                if (q0 + j < a.p && e < a.H) raw[j][v] = U::load(a.x[q0 + j], row * a.H + e);
            }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t e = (v * blockDim.x + threadIdx.x) * L;
                if (q0 + j < a.p && e < a.H) {
                    float x[L];
                    U::unpack(raw[j][v], x);
                    add_to<L>(h[v], x);
                }
            }
    }
}

// What the rows of a CTA share; each array for two rows in turn.
struct NormShared {
    float2 sum[2][32], again[2][32];
    uint32_t most[2][256];  // largest |y| of groups wider than a warp's units
};

// A row from its sum on: total, norm, 8 bits. w: the weight's units. n: threads that compute. False if any is bad.
template <int DT, int L, int V>
__device__ __forceinline__ bool finish_row(const NormArgs& a, size_t row, float (&h)[V][L], const typename Unit<DT, L>::Raw (&w)[V],
                                           NormShared& s, int turn, int n, bool bad) {
    using U = Unit<DT, L>;
    const auto at = [&](int v) { return (uint32_t(v) * n + threadIdx.x) * L; };
    // groups of fewer than 32 units are aligned lanes of one warp; in others a warp's 32 units, which start at a multiple of
    // 32 L, share a group
    const uint32_t H = uint32_t(a.H);
    const bool whole = a.shift < 0, narrow = !whole && (1 << a.shift) < 32 * L;
    if (a.has_q && !narrow)
        for (int i = threadIdx.x; i < 256; i += n) s.most[turn][i] = 0u;
    float ss = cta_sum2(dot<L, V>(h, h), 0.0f, s.sum[turn], n, bad).x;
    if (bad) return false;
    if (a.has_total)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (at(v) < H) store_all<DT, L>(a, a.total, row * a.H + at(v), h[v]);
    if (!(a.has_out || a.has_q)) return true;
    float eps = a.eps;
    if (ss == INFINITY) {  // the same for every thread
#pragma unroll
        for (int v = 0; v < V; ++v) mul_by<L>(h[v], kNormDown);
        ss = cta_sum2(dot<L, V>(h, h), 0.0f, s.again[turn], n, bad).x;
        eps = 0.0f;
    }
    const float r = 1.0f / sqrtf(ss / float(a.H) + eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (at(v) >= H) {
#pragma unroll
            for (int l = 0; l < L; ++l) h[v][l] = 0.0f;
            continue;
        }
        float f[L];
        U::unpack(w[v], f);
        mul_by<L>(h[v], r);
        mul_by<L>(h[v], f);
    }
    if (a.has_out)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (at(v) < H) store_all<DT, L>(a, a.out, row * a.H + at(v), h[v]);
    if (!a.has_q) return true;
    uint32_t most[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        most[v] = 0u;
#pragma unroll
        for (int l = 0; l < L; ++l) most[v] = max(most[v], magnitude(h[v][l]));
        if (narrow) {
            for (int d = (1 << a.shift) / L / 2; d > 0; d >>= 1) most[v] = max(most[v], __shfl_xor_sync(0xffffffffu, most[v], d));
        } else {
            most[v] = __reduce_max_sync(0xffffffffu, most[v]);
            if ((threadIdx.x & 31) == 0 && at(v) < H) atomicMax(&s.most[turn][whole ? 0 : at(v) >> a.shift], most[v]);
        }
    }
    if (!narrow) meet(n, false);
    const uint32_t groups = whole ? 1u : H >> a.shift;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (at(v) >= H) continue;
        const uint32_t g = whole ? 0u : at(v) >> a.shift;
        const float scale = scale_of(__uint_as_float(narrow ? most[v] : s.most[turn][g]));
#pragma unroll
        for (int l = 0; l < L; ++l) h[v][l] = over(h[v][l], scale);
        const typename Q8<L>::T q = Q8<L>::pack(h[v]);
#pragma unroll 4
        for (int k = a.rank0; k < a.rank0 + a.ranks; ++k) *reinterpret_cast<typename Q8<L>::T*>(a.q[k] + row * a.H + at(v)) = q;
        if (whole ? at(v) == 0 : (at(v) & ((1u << a.shift) - 1u)) == 0u)
            for (int k = a.rank0; k < a.rank0 + a.ranks; ++k) a.scale[k][row * groups + g] = scale;
    }
    return true;
}

// A row's gradient, and its share of the weight's. False if any thread is bad.
template <int DT, int L, int V>
__device__ __forceinline__ bool finish_grad(const NormArgs& a, size_t row, float (&h)[V][L], const float (&g)[V][L],
                                            const typename Unit<DT, L>::Raw (&past)[V], const float (&w)[V][L], float (&dw)[V][L],
                                            NormShared& s, int turn, int n, bool bad) {
    using U = Unit<DT, L>;
    const auto at = [&](int v) { return (uint32_t(v) * n + threadIdx.x) * L; };
    float wg[V][L];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int l = 0; l < L; ++l) wg[v][l] = g[v][l];
        mul_by<L>(wg[v], w[v]);
    }
    float2 sums = cta_sum2(dot<L, V>(h, h), dot<L, V>(wg, h), s.sum[turn], n, bad);
    if (bad) return false;
    float eps = a.eps, down = 1.0f;
    if (sums.x == INFINITY) {
        down = kNormDown;
        eps = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) mul_by<L>(h[v], down);
        sums = cta_sum2(dot<L, V>(h, h), dot<L, V>(wg, h), s.again[turn], n, bad);
    }
    const float r = 1.0f / sqrtf(sums.x / float(a.H) + eps), along = sums.y * r / float(a.H);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float away[L];
#pragma unroll
        for (int l = 0; l < L; ++l) away[l] = -along;
        mul_by<L>(h[v], r);  // u
        mul_add<L>(g[v], h[v], dw[v]);
        mul_add<L>(h[v], away, wg[v]);
        mul_by<L>(wg[v], r * down);
        if (at(v) >= a.H) continue;
        if (a.residual) {
            float add[L];
            U::unpack(past[v], add);
            add_to<L>(wg[v], add);
        }
        store_all<DT, L>(a, a.out, row * a.H + at(v), wg[v]);
    }
    return true;
}

// One row to a CTA, all its loads in registers.
template <int DT, int L, int V> __global__ void __launch_bounds__(V == 8 || L == 1 ? 1024 : 512)
k_rmsnorm(const __grid_constant__ NormArgs a) {
    using U = Unit<DT, L>;
    __shared__ NormShared s;
    const bool failed = status_failed(a.ctl);
    const size_t row = blockIdx.x;
    const auto at = [&](int v) { return (uint32_t(v) * blockDim.x + threadIdx.x) * L; };
    float h[V][L];
    typename U::Raw res[V], w[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (at(v) < a.H) {
            if (a.residual) res[v] = U::load(a.residual, row * a.H + at(v));
            if (a.has_out || a.has_q) w[v] = U::load(a.weight, at(v));
        }
    sum_ranks<DT, L, V>(a, row, h);
    if (a.residual)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (at(v) >= a.H) continue;
            float x[L];
            U::unpack(res[v], x);
            add_to<L>(h[v], x);
        }
    finish_row<DT, L, V>(a, row, h, w, s, 0, blockDim.x, failed);
}

// ---- rows through a ring -------------------------------------------------------------------------

// With many rows a CTA takes every gridDim-th. A warp of its own copies the ranks' rows, one after the other, into a ring
// of slots in shared memory (bulk copies, each completing on the slot's mbarrier), so that copies of this and the next
// rows are in flight whatever the other warps do; these add up a row from its slots and hand each back.
constexpr int kNormSlots = 32;

struct NormRing {
    NormShared s;
    uint64_t full[kNormSlots], empty[kNormSlots];
    uint32_t stop;  // the computing warps have given up
};

// The copying warp's one thread: source k of a row is rank k's, then the extra ones.
template <int DT> __device__ __forceinline__ void copy_rows(const NormArgs& a, NormRing& ring, unsigned char* slots, int n_slots, int sources,
                                                            const void* extra0, const void* extra1) {
    const uint32_t bytes = uint32_t(a.H * Elem<DT>::kBytes);
    uint32_t it = 0;
    bool ok = true;
    for (size_t row = blockIdx.x; row < a.T && ok; row += gridDim.x)
        for (int k = 0; k < sources && ok; ++k, ++it) {
            const uint32_t slot = it % n_slots, round = it / n_slots;
            if (round > 0) ok = mbar_wait_bounded(a.ctl, &ring.empty[slot], (round - 1) & 1, a.timeout_ns);
            if (*reinterpret_cast<volatile uint32_t*>(&ring.stop)) ok = false;
            if (!ok) break;
            const void* base = k < a.p ? a.x[k] : k == a.p ? extra0 : extra1;
            mbar_arrive_expect_tx(&ring.full[slot], bytes);
            bulk_g2s(slots + size_t(slot) * bytes, static_cast<const char*>(base) + row * bytes, bytes, &ring.full[slot]);
        }
    // the CTA stays until its copies have landed: the last n_slots of them
    for (uint32_t i = it > uint32_t(n_slots) ? it - n_slots : 0; i < it; ++i)
        mbar_wait_bounded(a.ctl, &ring.full[i % n_slots], (i / n_slots) & 1, kLandNs);
}

template <int DT, int V, bool GRAD> __global__ void __launch_bounds__(544, V == 1 ? 2 : 1) k_rmsnorm_ring(const __grid_constant__ NormArgs a, int n_slots) {
    constexpr int L = Pack16<DT>::L;
    using U = Unit<DT, L>;
    extern __shared__ __align__(128) unsigned char slots[];
    __shared__ NormRing ring;
    const int n = blockDim.x - 32;  // threads that compute
    if (threadIdx.x == 0) {
        for (int i = 0; i < n_slots; ++i) {
            mbar_init(&ring.full[i], 1);
            mbar_init(&ring.empty[i], n / 32);
        }
        ring.stop = 0u;
        fence_barrier_init();
    }
    if (__syncthreads_or(status_failed(a.ctl))) return;
    // the gradient has the rows h behind the ranks', and both forms the residual or what stands in its place
    const int sources = a.p + (GRAD ? 1 : 0) + (a.residual ? 1 : 0);
    if (int(threadIdx.x) >= n) {
        if (int(blockIdx.x) == a.fault_cta) return;  // fault injection
        if (int(threadIdx.x) == n) copy_rows<DT>(a, ring, slots, n_slots, sources, GRAD ? a.h : a.residual, a.residual);
        return;
    }
    const uint32_t bytes = uint32_t(a.H * Elem<DT>::kBytes);
    const auto at = [&](int v) { return (uint32_t(v) * n + threadIdx.x) * L; };
    typename U::Raw wr[V];
    float w[V][L], dw[V][L];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int l = 0; l < L; ++l) w[v][l] = dw[v][l] = 0.0f;
        if (at(v) < a.H && (GRAD || a.has_out || a.has_q)) {
            wr[v] = U::load(a.weight, at(v));
            if constexpr (GRAD) U::unpack(wr[v], w[v]);
        }
    }
    uint32_t slot = 0, phase = 0;
    bool bad = false;
    int turn = 0;
    // takes the next slot's units; every warp hands it back for itself
    auto take = [&](typename U::Raw (&raw)[V]) {
        if (!bad) bad = !mbar_wait_bounded(a.ctl, &ring.full[slot], phase, a.timeout_ns);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (!bad && at(v) < a.H) raw[v] = *reinterpret_cast<const uint4*>(slots + size_t(slot) * bytes + at(v) * Elem<DT>::kBytes);
        __syncwarp();
        if ((threadIdx.x & 31) == 0 && !bad) mbar_arrive(&ring.empty[slot]);
        if (++slot == uint32_t(n_slots)) {
            slot = 0;
            phase ^= 1;
        }
    };
    for (size_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        float sum[V][L];
        typename U::Raw raw[V], past[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            raw[v] = make_uint4(0, 0, 0, 0);  // stays where a thread has no unit
#pragma unroll
            for (int l = 0; l < L; ++l) sum[v][l] = -0.0f;  // the first addition leaves what it adds
        }
        for (int k = 0; k < a.p + (!GRAD && a.residual ? 1 : 0); ++k) {
            take(raw);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float x[L];
                U::unpack(raw[v], x);
                add_to<L>(sum[v], x);
            }
        }
        if constexpr (GRAD) {
            float h[V][L];
            take(raw);
#pragma unroll
            for (int v = 0; v < V; ++v) U::unpack(raw[v], h[v]);
            if (a.residual) take(past);
            if (!finish_grad<DT, L, V>(a, row, h, sum, past, w, dw, ring.s, turn, n, bad)) {
                ring.stop = 1u;
                return;
            }
        } else {
            if (!finish_row<DT, L, V>(a, row, sum, wr, ring.s, turn, n, bad)) {
                ring.stop = 1u;
                return;
            }
        }
    }
    if constexpr (GRAD) {
        if (!a.part) return;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int l = 0; l < L; ++l)
                if (at(v) < a.H) a.part[blockIdx.x * a.H + at(v) + l] = dw[v][l];
    }
}

// One element of the summed row.
template <int DT> __device__ __forceinline__ float sum_elem(const NormArgs& a, size_t at, bool residual) {
    float h = load_elem<DT>(a.x[0], at);
    for (int q = 1; q < a.p; ++q) h += load_elem<DT>(a.x[q], at);
    return residual ? h + load_elem<DT>(a.residual, at) : h;
}

// Any row: sums are formed again for each use. total is stored by the last use of an element, since a residual may be the
// same buffer.
template <int DT> __global__ void __launch_bounds__(1024) k_rmsnorm_long(const __grid_constant__ NormArgs a) {
    __shared__ float2 s_sum[32], s_again[32];
    __shared__ uint32_t s_most;
    bool bad = false;
    if (__syncthreads_or(status_failed(a.ctl))) return;
    const size_t row = blockIdx.x, o = row * a.H;
    const bool res = a.residual != nullptr, normed = a.has_out || a.has_q;
    float down = 1.0f, r = 0.0f;
    if (threadIdx.x == 0) s_most = 0u;
    if (normed) {
        float ss = 0.0f;
        for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) {
            const float h = sum_elem<DT>(a, o + i, res);
            ss += h * h;
        }
        ss = cta_sum2(ss, 0.0f, s_sum, blockDim.x, bad).x;
        float eps = a.eps;
        if (ss == INFINITY) {
            down = kNormDown;
            ss = 0.0f;
            for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) {
                const float h = sum_elem<DT>(a, o + i, res) * down;
                ss += h * h;
            }
            ss = cta_sum2(ss, 0.0f, s_again, blockDim.x, bad).x;
            eps = 0.0f;
        }
        r = 1.0f / sqrtf(ss / float(a.H) + eps);
    }
    auto norm = [&](float h, size_t i) { return h * down * r * load_elem<DT>(a.weight, i); };
    // stores what belongs to element i, its 8-bit value by the scale
    auto finish = [&](size_t i, float scale) {
        const float h = sum_elem<DT>(a, o + i, res), y = normed ? norm(h, i) : 0.0f;
        for (int k = a.rank0; k < a.rank0 + a.ranks; ++k) {
            if (a.has_total) store_elem<DT>(a.total[k], o + i, h);
            if (a.has_out) store_elem<DT>(a.out[k], o + i, y);
            if (a.has_q) a.q[k][o + i] = e4m3(over(y, scale));
        }
    };
    if (!a.has_q) {
        for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) finish(i, 0.0f);
        return;
    }
    const size_t groups = a.H / a.group;
    if (groups == 1) {
        uint32_t most = 0u;
        for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) most = max(most, magnitude(norm(sum_elem<DT>(a, o + i, res), i)));
        __syncthreads();
        atomicMax(&s_most, most);
        __syncthreads();
        const float scale = scale_of(__uint_as_float(s_most));
        if (threadIdx.x == 0)
            for (int k = a.rank0; k < a.rank0 + a.ranks; ++k) a.scale[k][row] = scale;
        for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) finish(i, scale);
        return;
    }
    const int lane = threadIdx.x & 31;
    for (size_t g = threadIdx.x >> 5; g < groups; g += blockDim.x >> 5) {  // a warp's groups
        uint32_t most = 0u;
        for (size_t i = g * a.group + lane; i < (g + 1) * a.group; i += 32) most = max(most, magnitude(norm(sum_elem<DT>(a, o + i, res), i)));
        const float scale = scale_of(__uint_as_float(__reduce_max_sync(0xffffffffu, most)));
        if (lane == 0)
            for (int k = a.rank0; k < a.rank0 + a.ranks; ++k) a.scale[k][row * groups + g] = scale;
        for (size_t i = g * a.group + lane; i < (g + 1) * a.group; i += 32) finish(i, scale);
    }
}

// ---- gradient ------------------------------------------------------------------------------------

template <int DT, int L, int V> __global__ void __launch_bounds__(V == 8 || L == 1 ? 1024 : 512)
k_rmsnorm_grad(const __grid_constant__ NormArgs a) {
    using U = Unit<DT, L>;
    __shared__ NormShared s;
    const bool failed = status_failed(a.ctl);
    const auto at = [&](int v) { return (uint32_t(v) * blockDim.x + threadIdx.x) * L; };
    float w[V][L], dw[V][L];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int l = 0; l < L; ++l) w[v][l] = dw[v][l] = 0.0f;
        if (at(v) < a.H) U::unpack(U::load(a.weight, at(v)), w[v]);
    }
    int turn = 0;
    for (size_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        float h[V][L], g[V][L];
        typename U::Raw hr[V], past[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (at(v) < a.H) {
                hr[v] = U::load(a.h, row * a.H + at(v));
                if (a.residual) past[v] = U::load(a.residual, row * a.H + at(v));
            }
        sum_ranks<DT, L, V>(a, row, g);
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int l = 0; l < L; ++l) h[v][l] = 0.0f;
            if (at(v) < a.H) U::unpack(hr[v], h[v]);
        }
        if (!finish_grad<DT, L, V>(a, row, h, g, past, w, dw, s, turn, blockDim.x, failed)) return;
    }
    if (!a.part) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int l = 0; l < L; ++l)
            if (at(v) < a.H) a.part[blockIdx.x * a.H + at(v) + l] = dw[v][l];
}

template <int DT> __global__ void __launch_bounds__(1024) k_rmsnorm_grad_long(const __grid_constant__ NormArgs a) {
    __shared__ float2 s_sum[2][32], s_again[2][32];
    bool bad = false;
    if (__syncthreads_or(status_failed(a.ctl))) return;
    int turn = 0;
    for (size_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const size_t o = row * a.H;
        float ss = 0.0f, wgh = 0.0f, eps = a.eps, down = 1.0f;
        auto add = [&](size_t i) {
            const float h = load_elem<DT>(a.h, o + i) * down;
            ss += h * h;
            wgh += load_elem<DT>(a.weight, i) * sum_elem<DT>(a, o + i, false) * h;
        };
        for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) add(i);
        float2 sums = cta_sum2(ss, wgh, s_sum[turn], blockDim.x, bad);
        if (sums.x == INFINITY) {
            down = kNormDown;
            ss = wgh = 0.0f;
            for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) add(i);
            sums = cta_sum2(ss, wgh, s_again[turn], blockDim.x, bad);
            eps = 0.0f;
        }
        const float r = 1.0f / sqrtf(sums.x / float(a.H) + eps), along = sums.y * r / float(a.H);
        for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) {
            const float u = load_elem<DT>(a.h, o + i) * down * r, g = sum_elem<DT>(a, o + i, false);
            float dx = (load_elem<DT>(a.weight, i) * g - u * along) * (r * down);
            if (a.residual) dx += load_elem<DT>(a.residual, o + i);
            for (int k = a.rank0; k < a.rank0 + a.ranks; ++k) store_elem<DT>(a.out[k], o + i, dx);
            if (a.part) {  // an element is one thread's in every row
                float* d = a.part + blockIdx.x * a.H + i;
                *d = row == blockIdx.x ? g * u : *d + g * u;
            }
        }
    }
}

// The weight's gradient: the CTAs' sums, each warp a share of them, then the shares in order. With 8 warps instead of 32 the
// sums of 296 CTAs for 4,096 columns took 8.3 us.
constexpr int kWeightWarps = 32;
__global__ void __launch_bounds__(32 * kWeightWarps) k_rmsnorm_grad_weight(const __grid_constant__ NormArgs a) {
    __shared__ float s_part[kWeightWarps][32];
    if (__syncthreads_or(status_failed(a.ctl))) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t i = size_t(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (i < a.H)
#pragma unroll 8
        for (int c = a.ctas * warp / kWeightWarps; c < a.ctas * (warp + 1) / kWeightWarps; ++c) s += __ldcg(a.part + c * a.H + i);
    s_part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || i >= a.H) return;
    for (int k = 1; k < kWeightWarps; ++k) s += s_part[k][lane];
    for (int k = a.rank0; k < a.rank0 + a.ranks; ++k) a.grad_weight[k][i] = s;
}

// How a row lies in a CTA: units of 16 bytes, 1 to 4 of them on up to 512 threads; single elements, 1, 2 or 8 to a thread, where
// rows are not whole vectors; or the kernels for any length. slots > 0: through a ring, per_sm CTAs to an SM.
struct NormShape {
    int form;     // 0: any length; 1, 2, 4: so many vectors to a thread; 11, 12, 18: 1, 2, 8 elements
    int threads;
    int slots, per_sm;
};
static NormShape norm_shape(const NormArgs& a, int dtype, bool grad, int num_sms) {
    const size_t L = dtype == COLL_BF16 ? 8 : 4, n = a.vec ? a.H / L : a.H;
    auto threads = [&](size_t per) { return int(((n + per - 1) / per + 31) / 32 * 32); };
    if (!a.vec) {
        if (n <= 256) return {11, threads(1), 0, 0};
        if (n <= 2048) return {12, threads(2), 0, 0};
        if (n <= 8192) return {18, threads(8), 0, 0};
        return {0, 1024, 0, 0};
    }
    if (n > 2048) return {0, 1024, 0, 0};
    const int V = n <= 512 ? 1 : n <= 1024 ? 2 : 4;
    NormShape s{V, threads(V), 0, 0};
    // A ring pays where a row is long and each CTA has some. Measured on B200, 8 ranks bf16, us with the ring and without: 592
    // rows of 4096 23 and 27 (gradient 31 and 32), of 8192 43 and 47 (49 and 53); 296 rows alike; 4800 rows of 2048 89 and 91
    // (90 and 77), of 1024 47 and 42 (50 and 57), of 256 32 and 13 (44 and 42). Two CTAs of one vector to a thread fit an SM by
    // their registers, and one forms its sums while the other stores (2048 rows of 4096 in 8 bits 66 us, with one 79).
    s.per_sm = V > 1 ? 1 : 2;
    const size_t bytes = n * 16, slots = std::min<size_t>(kNormSlots, (size_t(220) * 1024 / s.per_sm - 8192) / bytes);
    if (n >= 512 && slots >= 4 && !(grad && V == 4) && a.T >= size_t(2 * num_sms * s.per_sm)) s.slots = int(slots);
    return s;
}
static int ring_ctas(const NormArgs& a, const NormShape& n, int num_sms) { return int(std::min(a.T, size_t(num_sms * n.per_sm))); }

// CTAs of the gradient: each one's sums of the weight's gradient are H numbers of scratch.
int rmsnorm_grad_ctas(const NormArgs& a, int dtype, int num_sms) {
    const NormShape n = norm_shape(a, dtype, true, num_sms);
    return n.slots ? ring_ctas(a, n, num_sms) : int(std::min(a.T, size_t(num_sms) * std::max(1, 512 / n.threads)));
}

template <int DT, int V, bool GRAD> static cudaError_t go_ring(const NormArgs& a, const NormShape& n, int ctas, cudaStream_t s) {
    const size_t smem = size_t(n.slots) * a.H * Elem<DT>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(k_rmsnorm_ring<DT, V, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    k_rmsnorm_ring<DT, V, GRAD><<<ctas, n.threads + 32, smem, s>>>(a, n.slots);
    return cudaGetLastError();
}

template <int DT> static cudaError_t go_norm(const NormArgs& a, const NormShape& n, int num_sms, cudaStream_t s) {
    constexpr int L = Pack16<DT>::L;
    const unsigned ctas = unsigned(a.T);
    if (n.slots) {
        const int c = ring_ctas(a, n, num_sms);
        return n.form == 1 ? go_ring<DT, 1, false>(a, n, c, s) : n.form == 2 ? go_ring<DT, 2, false>(a, n, c, s) : go_ring<DT, 4, false>(a, n, c, s);
    }
    switch (n.form) {
        case 1: k_rmsnorm<DT, L, 1><<<ctas, n.threads, 0, s>>>(a); break;
        case 2: k_rmsnorm<DT, L, 2><<<ctas, n.threads, 0, s>>>(a); break;
        case 4: k_rmsnorm<DT, L, 4><<<ctas, n.threads, 0, s>>>(a); break;
        case 11: k_rmsnorm<DT, 1, 1><<<ctas, n.threads, 0, s>>>(a); break;
        case 12: k_rmsnorm<DT, 1, 2><<<ctas, n.threads, 0, s>>>(a); break;
        case 18: k_rmsnorm<DT, 1, 8><<<ctas, n.threads, 0, s>>>(a); break;
        default: k_rmsnorm_long<DT><<<ctas, n.threads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <int DT> static cudaError_t go_norm_grad(const NormArgs& a, const NormShape& n, cudaStream_t s) {
    constexpr int L = Pack16<DT>::L;
    const unsigned ctas = unsigned(a.ctas);
    if (n.slots) return n.form == 1 ? go_ring<DT, 1, true>(a, n, a.ctas, s) : go_ring<DT, 2, true>(a, n, a.ctas, s);
    switch (n.form) {
        case 1: k_rmsnorm_grad<DT, L, 1><<<ctas, n.threads, 0, s>>>(a); break;
        case 2: k_rmsnorm_grad<DT, L, 2><<<ctas, n.threads, 0, s>>>(a); break;
        case 4: k_rmsnorm_grad<DT, L, 4><<<ctas, n.threads, 0, s>>>(a); break;
        case 11: k_rmsnorm_grad<DT, 1, 1><<<ctas, n.threads, 0, s>>>(a); break;
        case 12: k_rmsnorm_grad<DT, 1, 2><<<ctas, n.threads, 0, s>>>(a); break;
        case 18: k_rmsnorm_grad<DT, 1, 8><<<ctas, n.threads, 0, s>>>(a); break;
        default: k_rmsnorm_grad_long<DT><<<ctas, n.threads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_rmsnorm(const NormArgs& a, int dtype, int num_sms, cudaStream_t s) {
    if (a.T > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    const NormShape n = norm_shape(a, dtype, false, num_sms);
    return dtype == COLL_BF16 ? go_norm<COLL_BF16>(a, n, num_sms, s) : go_norm<COLL_FP32>(a, n, num_sms, s);
}

cudaError_t launch_rmsnorm_grad(const NormArgs& a, int dtype, int num_sms, cudaStream_t s, int* kernels_launched) {
    const NormShape n = norm_shape(a, dtype, true, num_sms);
    cudaError_t e = dtype == COLL_BF16 ? go_norm_grad<COLL_BF16>(a, n, s) : go_norm_grad<COLL_FP32>(a, n, s);
    *kernels_launched = 1;
    if (e != cudaSuccess || !a.part) return e;
    k_rmsnorm_grad_weight<<<unsigned((a.H + 31) / 32), 32 * kWeightWarps, 0, s>>>(a);
    *kernels_launched = 2;
    return cudaGetLastError();
}

}  // namespace simcomm
