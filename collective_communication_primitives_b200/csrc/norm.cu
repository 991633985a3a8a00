// Root-mean-square norm of rows that lie on the ranks as partial sums, with the AllReduce before it, the residual's
// addition and 8-bit rows; and its gradient.
//
//   h = sum_q x[q] + residual,  y = h w r,  r = 1 / sqrt(mean h^2 + eps);  8 bits: scale = max |y| / 448 per group, q = y / scale
//   gradient, g = sum_q grad_out[q]:  u = h r,  dh = r (w g - u mean(w g u)) + grad_total,  dw = sum over rows of g u
//
// One CTA has a row. Its threads keep the sum of all ranks' partial rows in registers, so that every input is read once,
// and write the finished row to every rank: p + 1 rows in, p (2 bytes or more) rows out. Bound by these bytes; for a few
// rows by the latency of one load, one reduction and one store. Rows too long for registers are summed again for
// each use.
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
    __device__ static void store(void* base, size_t e, const float (&a)[L]) {
        st_v4(static_cast<char*>(base) + e * D, Pack16<DT>::pack(a));
    }
};
template <int DT> struct Unit<DT, 1> {
    using Raw = float;
    __device__ static Raw load(const void* base, size_t e) { return load_elem<DT>(base, e); }
    __device__ static void unpack(const Raw& v, float (&a)[1]) { a[0] = v; }
    __device__ static void store(void* base, size_t e, const float (&a)[1]) { store_elem<DT>(base, e, a[0]); }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
// The CTA's sums of two values per thread, in a fixed order, the same for every thread. buf: 2 x 32, free to be
// written again after another barrier.
__device__ __forceinline__ float2 cta_sum2(float a, float b, float2* buf) {
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    a = warp_sum(a);
    b = warp_sum(b);
    if (lane == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 v = lane < warps ? buf[lane] : make_float2(0.0f, 0.0f);
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
template <int L> __device__ __forceinline__ void store_q(uint8_t* p, const float (&v)[L]) {
    if constexpr (L == 1) {
        *p = e4m3(v[0]);
    } else {
        uint32_t w[L / 4];
#pragma unroll
        for (int i = 0; i < L / 4; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
        if constexpr (L == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(p) = w[0];
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
        for (int l = 0; l < L; ++l) h[v][l] = 0.0f;
    for (int q0 = 0; q0 < a.p; q0 += kAhead) {
        typename U::Raw raw[kAhead][V];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const size_t e = (size_t(v) * blockDim.x + threadIdx.x) * L;
                if (q0 + j < a.p && e < a.H) raw[j][v] = U::load(a.x[q0 + j], row * a.H + e);
            }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const size_t e = (size_t(v) * blockDim.x + threadIdx.x) * L;
                if (q0 + j < a.p && e < a.H) {
                    float x[L];
                    U::unpack(raw[j][v], x);
#pragma unroll
                    for (int l = 0; l < L; ++l) h[v][l] = q0 + j == 0 ? x[l] : h[v][l] + x[l];
                }
            }
    }
}

template <int DT, int L, int V> __global__ void __launch_bounds__(V == 8 ? 1024 : 512)
k_rmsnorm(const __grid_constant__ NormArgs a) {
    using U = Unit<DT, L>;
    __shared__ float2 s_sum[32], s_again[32];
    __shared__ uint32_t s_most[256];  // largest |y| of groups wider than a warp's units
    const bool failed = status_failed(a.ctl);
    const size_t row = blockIdx.x;
    // groups of fewer than 32 units are aligned lanes of one warp; in others a warp's 32 units, which start at a multiple of
    // 32 L, share a group
    const bool narrow = a.has_q && size_t(a.group) < size_t(32 * L) && size_t(a.group) < a.H;
    const bool whole = a.has_q && !narrow && size_t(a.group) == a.H;
    if (a.has_q && !narrow)
        for (int i = threadIdx.x; i < 256; i += blockDim.x) s_most[i] = 0u;
    float h[V][L], w[V][L];
    const auto at = [&](int v) { return (size_t(v) * blockDim.x + threadIdx.x) * L; };
    typename U::Raw res[V], wr[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (at(v) < a.H) {
            if (a.residual) res[v] = U::load(a.residual, row * a.H + at(v));
            if (a.has_out || a.has_q) wr[v] = U::load(a.weight, at(v));
        }
    sum_ranks<DT, L, V>(a, row, h);
    if (__syncthreads_or(failed)) return;
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool in = at(v) < a.H;
        if (in && a.residual) {
            float x[L];
            U::unpack(res[v], x);
#pragma unroll
            for (int l = 0; l < L; ++l) h[v][l] += x[l];
        }
        if (in && (a.has_out || a.has_q)) U::unpack(wr[v], w[v]);
#pragma unroll
        for (int l = 0; l < L; ++l) ss += h[v][l] * h[v][l];
        if (in && a.has_total)
            for (int r = a.rank0; r < a.rank0 + a.ranks; ++r) U::store(a.total[r], row * a.H + at(v), h[v]);
    }
    if (!(a.has_out || a.has_q)) return;
    ss = cta_sum2(ss, 0.0f, s_sum).x;
    float eps = a.eps;
    if (ss == INFINITY) {  // the same for every thread
        ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int l = 0; l < L; ++l) {
                h[v][l] *= kNormDown;
                ss += h[v][l] * h[v][l];
            }
        ss = cta_sum2(ss, 0.0f, s_again).x;
        eps = 0.0f;
    }
    const float r = 1.0f / sqrtf(ss / float(a.H) + eps);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int l = 0; l < L; ++l) h[v][l] = at(v) < a.H ? h[v][l] * r * w[v][l] : 0.0f;
    if (a.has_out)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (at(v) < a.H)
                for (int r2 = a.rank0; r2 < a.rank0 + a.ranks; ++r2) U::store(a.out[r2], row * a.H + at(v), h[v]);
    if (!a.has_q) return;
    uint32_t most[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        most[v] = 0u;
#pragma unroll
        for (int l = 0; l < L; ++l) most[v] = max(most[v], magnitude(h[v][l]));
        if (narrow) {
            for (int d = a.group / L / 2; d > 0; d >>= 1) most[v] = max(most[v], __shfl_xor_sync(0xffffffffu, most[v], d));
        } else {
            most[v] = __reduce_max_sync(0xffffffffu, most[v]);
            if ((threadIdx.x & 31) == 0 && at(v) < a.H) atomicMax(&s_most[whole ? 0 : at(v) / a.group], most[v]);
        }
    }
    if (!narrow) __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (at(v) >= a.H) continue;
        const size_t g = whole ? 0 : at(v) / a.group;
        const float scale = scale_of(__uint_as_float(narrow ? most[v] : s_most[g]));
#pragma unroll
        for (int l = 0; l < L; ++l) h[v][l] = over(h[v][l], scale);
        const bool first = whole ? at(v) == 0 : at(v) % a.group == 0;
        for (int r2 = a.rank0; r2 < a.rank0 + a.ranks; ++r2) {
            store_q<L>(a.q[r2] + row * a.H + at(v), h[v]);
            if (first) a.scale[r2][row * (a.H / a.group) + g] = scale;
        }
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
        ss = cta_sum2(ss, 0.0f, s_sum).x;
        float eps = a.eps;
        if (ss == INFINITY) {
            down = kNormDown;
            ss = 0.0f;
            for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) {
                const float h = sum_elem<DT>(a, o + i, res) * down;
                ss += h * h;
            }
            ss = cta_sum2(ss, 0.0f, s_again).x;
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

template <int DT, int L, int V> __global__ void __launch_bounds__(V == 8 ? 1024 : 512)
k_rmsnorm_grad(const __grid_constant__ NormArgs a) {
    using U = Unit<DT, L>;
    __shared__ float2 s_sum[2][32], s_again[32];
    if (__syncthreads_or(status_failed(a.ctl))) return;
    const auto at = [&](int v) { return (size_t(v) * blockDim.x + threadIdx.x) * L; };
    float w[V][L], dw[V][L];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int l = 0; l < L; ++l) w[v][l] = dw[v][l] = 0.0f;
        if (at(v) < a.H) U::unpack(U::load(a.weight, at(v)), w[v]);
    }
    int turn = 0;
    for (size_t row = blockIdx.x; row < a.T; row += a.ctas, turn ^= 1) {
        float h[V][L], g[V][L];
        typename U::Raw hr[V], past[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (at(v) < a.H) {
                hr[v] = U::load(a.h, row * a.H + at(v));
                if (a.residual) past[v] = U::load(a.residual, row * a.H + at(v));
            }
        sum_ranks<DT, L, V>(a, row, g);
        float ss = 0.0f, wgh = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int l = 0; l < L; ++l) h[v][l] = 0.0f;
            if (at(v) < a.H) U::unpack(hr[v], h[v]);
#pragma unroll
            for (int l = 0; l < L; ++l) {
                ss += h[v][l] * h[v][l];
                wgh += w[v][l] * g[v][l] * h[v][l];
            }
        }
        // the buffers alternate: the next row's are written after this row's barrier, which no thread passes that
        // still reads the row's before
        float2 sums = cta_sum2(ss, wgh, s_sum[turn]);
        float eps = a.eps, down = 1.0f;
        if (sums.x == INFINITY) {
            down = kNormDown;
            ss = wgh = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int l = 0; l < L; ++l) {
                    h[v][l] *= down;
                    ss += h[v][l] * h[v][l];
                    wgh += w[v][l] * g[v][l] * h[v][l];
                }
            sums = cta_sum2(ss, wgh, s_again);
            __syncthreads();
            eps = 0.0f;
        }
        const float r = 1.0f / sqrtf(sums.x / float(a.H) + eps), along = sums.y * r / float(a.H);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float dx[L], add[L];
#pragma unroll
            for (int l = 0; l < L; ++l) {
                const float u = h[v][l] * r;
                dw[v][l] += g[v][l] * u;
                dx[l] = (w[v][l] * g[v][l] - u * along) * (r * down);
            }
            if (at(v) >= a.H) continue;
            if (a.residual) {
                U::unpack(past[v], add);
#pragma unroll
                for (int l = 0; l < L; ++l) dx[l] += add[l];
            }
            for (int k = a.rank0; k < a.rank0 + a.ranks; ++k) U::store(a.out[k], row * a.H + at(v), dx);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int l = 0; l < L; ++l)
            if (at(v) < a.H) a.part[blockIdx.x * a.H + at(v) + l] = dw[v][l];
}

template <int DT> __global__ void __launch_bounds__(1024) k_rmsnorm_grad_long(const __grid_constant__ NormArgs a) {
    __shared__ float2 s_sum[2][32], s_again[32];
    if (__syncthreads_or(status_failed(a.ctl))) return;
    int turn = 0;
    for (size_t row = blockIdx.x; row < a.T; row += a.ctas, turn ^= 1) {
        const size_t o = row * a.H;
        float ss = 0.0f, wgh = 0.0f, eps = a.eps, down = 1.0f;
        auto add = [&](size_t i) {
            const float h = load_elem<DT>(a.h, o + i) * down;
            ss += h * h;
            wgh += load_elem<DT>(a.weight, i) * sum_elem<DT>(a, o + i, false) * h;
        };
        for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) add(i);
        float2 sums = cta_sum2(ss, wgh, s_sum[turn]);
        if (sums.x == INFINITY) {
            down = kNormDown;
            ss = wgh = 0.0f;
            for (size_t i = threadIdx.x; i < a.H; i += blockDim.x) add(i);
            sums = cta_sum2(ss, wgh, s_again);
            __syncthreads();
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

// The weight's gradient: the CTAs' sums, 8 warps each an eighth of them, then the eighths in order.
__global__ void __launch_bounds__(256) k_rmsnorm_grad_weight(const __grid_constant__ NormArgs a) {
    __shared__ float s_part[8][32];
    if (__syncthreads_or(status_failed(a.ctl))) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t i = size_t(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (i < a.H)
#pragma unroll 8
        for (int c = a.ctas * warp / 8; c < a.ctas * (warp + 1) / 8; ++c) s += __ldcg(a.part + c * a.H + i);
    s_part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || i >= a.H) return;
    for (int k = 1; k < 8; ++k) s += s_part[k][lane];
    for (int k = a.rank0; k < a.rank0 + a.ranks; ++k) a.grad_weight[k][i] = s;
}

// CTAs of the gradient, whatever the row's length: each one's sums of the weight's gradient are H numbers of scratch.
int rmsnorm_grad_ctas(size_t rows, int num_sms) { return int(std::min(rows, size_t(num_sms) * 2)); }

// How a row lies in a CTA: units of 16 bytes, 1 to 4 of them on up to 1024 threads; single elements, 1 or 8 to a thread, where rows
// are not whole vectors; or the kernels for any length.
struct NormShape {
    int form;     // 0: any length, 1: 1 vector, 2: 2, 4: 4 vectors, 11: 1 element, 18: 8 elements
    int threads;
};
static NormShape norm_shape(const NormArgs& a, int dtype) {
    const size_t L = dtype == COLL_BF16 ? 8 : 4, n = a.vec ? a.H / L : a.H;
    auto threads = [&](size_t per) { return int(((n + per - 1) / per + 31) / 32 * 32); };
    if (a.vec) {
        if (n <= 512) return {1, threads(1)};
        if (n <= 1024) return {2, threads(2)};
        if (n <= 2048) return {4, threads(4)};
        return {0, 1024};
    }
    if (n <= 256) return {11, threads(1)};
    if (n <= 8192) return {18, threads(8)};
    return {0, 1024};
}

template <int DT> static void go_norm(const NormArgs& a, const NormShape& n, unsigned ctas, cudaStream_t s) {
    constexpr int L = Pack16<DT>::L;
    switch (n.form) {
        case 1: k_rmsnorm<DT, L, 1><<<ctas, n.threads, 0, s>>>(a); break;
        case 2: k_rmsnorm<DT, L, 2><<<ctas, n.threads, 0, s>>>(a); break;
        case 4: k_rmsnorm<DT, L, 4><<<ctas, n.threads, 0, s>>>(a); break;
        case 11: k_rmsnorm<DT, 1, 1><<<ctas, n.threads, 0, s>>>(a); break;
        case 18: k_rmsnorm<DT, 1, 8><<<ctas, n.threads, 0, s>>>(a); break;
        default: k_rmsnorm_long<DT><<<ctas, n.threads, 0, s>>>(a);
    }
}

template <int DT> static void go_norm_grad(const NormArgs& a, const NormShape& n, cudaStream_t s) {
    constexpr int L = Pack16<DT>::L;
    const unsigned ctas = unsigned(a.ctas);
    switch (n.form) {
        case 1: k_rmsnorm_grad<DT, L, 1><<<ctas, n.threads, 0, s>>>(a); break;
        case 2: k_rmsnorm_grad<DT, L, 2><<<ctas, n.threads, 0, s>>>(a); break;
        case 4: k_rmsnorm_grad<DT, L, 4><<<ctas, n.threads, 0, s>>>(a); break;
        case 11: k_rmsnorm_grad<DT, 1, 1><<<ctas, n.threads, 0, s>>>(a); break;
        case 18: k_rmsnorm_grad<DT, 1, 8><<<ctas, n.threads, 0, s>>>(a); break;
        default: k_rmsnorm_grad_long<DT><<<ctas, n.threads, 0, s>>>(a);
    }
}

cudaError_t launch_rmsnorm(const NormArgs& a, int dtype, cudaStream_t s) {
    if (a.T > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    const NormShape n = norm_shape(a, dtype);
    if (dtype == COLL_BF16) go_norm<COLL_BF16>(a, n, unsigned(a.T), s);
    else go_norm<COLL_FP32>(a, n, unsigned(a.T), s);
    return cudaGetLastError();
}

cudaError_t launch_rmsnorm_grad(const NormArgs& a, int dtype, cudaStream_t s, int* kernels_launched) {
    const NormShape n = norm_shape(a, dtype);
    if (dtype == COLL_BF16) go_norm_grad<COLL_BF16>(a, n, s);
    else go_norm_grad<COLL_FP32>(a, n, s);
    *kernels_launched = 1;
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.part) return e;
    k_rmsnorm_grad_weight<<<unsigned((a.H + 31) / 32), 256, 0, s>>>(a);
    *kernels_launched = 2;
    return cudaGetLastError();
}

}  // namespace simcomm
