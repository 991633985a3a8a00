// How the operators on scores go through a row whose V columns are sharded over the ranks: rank r holds columns [r m,
// (r+1) m), m = ceil(V / p), in logits[r] [rows][ld]. Args has logits, m and ld.
#pragma once

#include "common.cuh"

namespace simcomm {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpUnroll = 4;            // 16-byte loads in flight per thread
constexpr float kLpLog2e = 1.4426950408889634f;
constexpr float kLpLn2 = 0.6931471805599453f;

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

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The largest of a 16-byte vector of scores, NaN if any is.
template <int DT> __device__ __forceinline__ float vector_top(const uint4& v) {
    if constexpr (DT == COLL_BF16) {
        const uint32_t p = max_nan_bf16x2(max_nan_bf16x2(v.x, v.y), max_nan_bf16x2(v.z, v.w));
        return max_nan(bf16_bits_to_float(p), __uint_as_float(p & 0xffff0000u));
    } else {
        return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
}

// A shard's part of the columns [v, v1): how it lies in vectors.
template <int DT> struct Piece {
    static constexpr int L = Pack16<DT>::L, D = Elem<DT>::kBytes;
    const char* base;             // column v
    uint32_t end;                 // the next piece's first column
    uint32_t head, vecs, tail;    // scores before the first whole vector, vectors, scores after the last
    template <typename Args> __device__ __forceinline__ Piece(const Args& a, size_t row, uint32_t v, uint32_t v1) {
        const uint32_t m = uint32_t(a.m), r = v / m;  // a vocabulary has fewer than 2^31 columns
        end = min(v1, (r + 1) * m);
        base = static_cast<const char*>(a.logits[r]) + (row * a.ld + (v - r * m)) * D;
        const uint32_t n = end - v;
        head = min(n, uint32_t((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / D);
        vecs = (n - head) / L;
        tail = n - head - vecs * L;
    }
    __device__ __forceinline__ const char* vector(uint32_t i) const { return base + size_t(head) * D + size_t(i) * 16; }
    // Score k of the head + tail at the ends, and its place in the piece.
    __device__ __forceinline__ uint32_t end_at(uint32_t k) const { return k < head ? k : k + vecs * L; }
};

// Calls take(raw vector, scores in it, column of the first) for all columns [v0, v1) of a row; vector i of a
// piece falls to thread i modulo kLpThreads. Scores at the ends of pieces come as vectors of one score, one per
// lane of the first warp; missing scores are -inf. batch(raw vectors, whether they are the warp's
// first) comes before the vectors are taken.
template <int DT, typename Args, typename Take, typename Batch>
__device__ __forceinline__ void scan_columns(const Args& a, size_t row, uint32_t v0, uint32_t v1, Take take, Batch batch) {
    constexpr int L = Pack16<DT>::L;
    constexpr uint32_t kNone = DT == COLL_BF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
    const uint32_t warp0 = threadIdx.x & ~31u;
    for (uint32_t v = v0; v < v1;) {
        const Piece<DT> pc(a, row, v, v1);
        if (pc.head + pc.tail && threadIdx.x < 32) {
            const int cnt = threadIdx.x < pc.head + pc.tail ? 1 : 0;
            const uint32_t at = pc.end_at(threadIdx.x);
            uint4 raw = make_uint4(kNone, kNone, kNone, kNone);
            if (cnt) {
                if constexpr (DT == COLL_BF16) raw.x = (kNone & 0xffff0000u) | reinterpret_cast<const uint16_t*>(pc.base)[at];
                else raw.x = reinterpret_cast<const uint32_t*>(pc.base)[at];
            }
            const uint4 none = make_uint4(kNone, kNone, kNone, kNone), ends[kLpUnroll] = {raw, none, none, none};
            batch(ends, false);
            take(raw, cnt, v + at);
        }
        for (uint32_t i0 = 0; i0 < pc.vecs; i0 += kLpThreads * kLpUnroll) {
            uint4 raw[kLpUnroll];
#pragma unroll
            for (int q = 0; q < kLpUnroll; ++q) {
                const uint32_t i = i0 + q * kLpThreads + threadIdx.x;
                raw[q] = i < pc.vecs ? ld_stream_v4(pc.vector(i)) : make_uint4(kNone, kNone, kNone, kNone);
            }
            batch(raw, i0 == 0 && v == v0);
#pragma unroll
            for (int q = 0; q < kLpUnroll; ++q) {
                const uint32_t i = i0 + q * kLpThreads + threadIdx.x;
                if (i0 + q * kLpThreads + warp0 >= pc.vecs) break;  // none of this warp's
                take(raw[q], i < pc.vecs ? L : 0, v + pc.head + i * L);
            }
        }
        v = pc.end;
    }
}

template <typename Args> __device__ __forceinline__ float score_at(const Args& a, int dtype, size_t row, size_t v) {
    const size_t r = v / a.m, at = row * a.ld + (v - r * a.m);
    return dtype == COLL_BF16 ? load_elem<COLL_BF16>(a.logits[r], at) : load_elem<COLL_FP32>(a.logits[r], at);
}

// The CTA's sum of one value per thread, in a fixed order; the same for every thread.
template <typename T> __device__ __forceinline__ T cta_sum(T v, T* s_w) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = v;
    __syncthreads();
    T t = 0;
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

}  // namespace simcomm
