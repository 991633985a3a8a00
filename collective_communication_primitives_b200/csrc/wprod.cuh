// Products of a weight matrix with few tokens, streamed: the device code that the 4-bit linear and
// the expert layer share.
//
//   D[r][n] = sum_k W[r][k] X[n][k],   16 weight rows x 8 NT tokens per warp
//
// With few tokens the weights' bytes bound the time: every weight is used once per token, so the job
// is to keep enough 16-byte loads in flight and to spend few instructions per byte. The weights go
// from memory straight into the registers of the matrix instruction (mma.sync m16n8k16, weights as
// its 16-row operand and tokens as its 8 columns, so that one token wastes no more than 7 columns):
// no pass through shared memory. That works because a sum over k may be taken in any order as long
// as both operands use the same one: lane (g, t) (g = lane / 4, t = lane % 4) of the instruction owns
// rows g and g + 8 and four k's of every step, so it is given 8 consecutive k's of both rows, one
// 16-byte load each for bf16, and the tokens' lanes load the same k's of their rows. A step of the
// warp ("chunk") covers 32 k's of bf16 weights, or 8 LW x 4 of 4-bit ones, LW words of eight weights
// per lane, so that a chunk never crosses a scale group.
//
// 4-bit weights: word bits 4i..4i+3 hold weight i of eight, value q - 8. (w & 0x000F000F) | 0x43004300
// is the pair (128 + q_0, 128 + q_4) of bf16 values, and subtracting 136 is exact; shifts by 4 give
// the pairs (1,5), (2,6), (3,7), and the tokens' words are paired the same way. A chunk's sum is
// taken over the whole numbers q - 8 (bf16 holds them, the products are exact in fp32) and scaled
// once per chunk in fp32, so the weights are never rounded.
//
// Sums are held in fp32 throughout: the matrix instruction's accumulator, then plain adds over the
// warps that share a row tile, in warp order.
#pragma once

#include "common.cuh"

namespace simcomm {

enum WeightKind { W_BF16 = 0, W_Q4X4 = 1, W_Q4X2 = 2, W_Q4X1 = 3 };

template <int WK> struct WTraits {
    static constexpr bool kQ4 = WK != W_BF16;
    static constexpr int kWords = WK == W_Q4X4 ? 4 : WK == W_Q4X2 ? 2 : WK == W_Q4X1 ? 1 : 0;  // 4-bit: words per lane
    static constexpr int kLaneK = kQ4 ? 8 * kWords : 8;  // k's of one lane in a chunk
    static constexpr int kChunk = 4 * kLaneK;            // k's of a warp's chunk
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights are read once: streaming loads that leave L1 to the tokens.
__device__ __forceinline__ uint2 ld_stream_v2(const void* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_stream_u32(const void* p) {
    uint32_t v;
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// Eight consecutive bf16 values from element k of a row of K, zero past the end. VEC: K and the row
// are multiples of 16 bytes; otherwise one element at a time.
template <bool VEC> __device__ __forceinline__ uint4 ld_row8(const uint16_t* row, int k, int K) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (!row || k >= K) return v;
    if constexpr (VEC) {
        return *reinterpret_cast<const uint4*>(row + k);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = row[k + 2 * i < K ? k + 2 * i : k], hi = row[k + 2 * i + 1 < K ? k + 2 * i + 1 : k];
            w[i] = (k + 2 * i < K ? lo : 0u) | (k + 2 * i + 1 < K ? hi << 16 : 0u);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <bool VEC> __device__ __forceinline__ uint4 ld_weight8(const uint16_t* row, int k, int K) {
    if constexpr (VEC) return (row && k < K) ? ld_stream_v4(row + k) : make_uint4(0u, 0u, 0u, 0u);
    else return ld_row8<false>(row, k, K);
}

// Two bf16 values q - 8 of the nibble pair (i, i + 4) of a word shifted right by 4 i.
__device__ __forceinline__ uint32_t q4_pair(uint32_t w) {
    const uint32_t biased = (w & 0x000F000Fu) | 0x43004300u;
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(biased), "r"(0x43084308u));
    return r;
}

// One lane's view of a warp's product: rows g and g + 8 of the row tile and NT token rows.
struct LaneRows {
    const char* w0;          // weight row g (null: past the matrix, reads as zero)
    const char* w1;          // weight row g + 8
    const uint16_t* s0;      // 4-bit: scales of the rows, one per group
    const uint16_t* s1;
};

// acc += the product over chunks [c0, c1) of a row of K.
template <int WK, bool VEC, int NT>
__device__ __forceinline__ void warp_product(float (&acc)[NT][4], const LaneRows& r, const uint16_t* const (&x)[NT],
                                             int c0, int c1, int K, int groups_per_chunk_shift, int t) {
    using W = WTraits<WK>;
    if constexpr (!W::kQ4) {
        constexpr int U = 4;  // chunks in flight per lane
        const uint16_t* w0 = reinterpret_cast<const uint16_t*>(r.w0);
        const uint16_t* w1 = reinterpret_cast<const uint16_t*>(r.w1);
        for (int c = c0; c < c1; c += U) {
            uint4 a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = c + u < c1 ? (c + u) * W::kChunk + t * 8 : K;
                a[u] = ld_weight8<VEC>(w0, k, K);
                b[u] = ld_weight8<VEC>(w1, k, K);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = c + u < c1 ? (c + u) * W::kChunk + t * 8 : K;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 xv = ld_row8<VEC>(x[n], k, K);
                    mma_bf16(acc[n], a[u].x, b[u].x, a[u].y, b[u].y, xv.x, xv.y);
                    mma_bf16(acc[n], a[u].z, b[u].z, a[u].w, b[u].w, xv.z, xv.w);
                }
            }
        }
    } else {
        constexpr int U = W::kWords == 4 ? 4 : W::kWords == 2 ? 8 : 8;
        for (int c = c0; c < c1; c += U) {
            uint32_t a[U][W::kWords], b[U][W::kWords];
            float sa[U], sb[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = c + u < c1;
                const size_t off = (size_t(c + u) * 4 + t) * (4 * W::kWords);
                const int grp = (c + u) >> groups_per_chunk_shift;
#pragma unroll
                for (int j = 0; j < W::kWords; ++j) a[u][j] = b[u][j] = 0u;
                sa[u] = sb[u] = 0.0f;
                if (in && r.w0) {
                    if constexpr (W::kWords == 4) {
                        const uint4 v = ld_stream_v4(r.w0 + off);
                        a[u][0] = v.x; a[u][1] = v.y; a[u][2] = v.z; a[u][3] = v.w;
                    } else if constexpr (W::kWords == 2) {
                        const uint2 v = ld_stream_v2(r.w0 + off);
                        a[u][0] = v.x; a[u][1] = v.y;
                    } else a[u][0] = *reinterpret_cast<const uint32_t*>(r.w0 + off);
                    sa[u] = bf16_bits_to_float(r.s0[grp]);
                }
                if (in && r.w1) {
                    if constexpr (W::kWords == 4) {
                        const uint4 v = ld_stream_v4(r.w1 + off);
                        b[u][0] = v.x; b[u][1] = v.y; b[u][2] = v.z; b[u][3] = v.w;
                    } else if constexpr (W::kWords == 2) {
                        const uint2 v = ld_stream_v2(r.w1 + off);
                        b[u][0] = v.x; b[u][1] = v.y;
                    } else b[u][0] = *reinterpret_cast<const uint32_t*>(r.w1 + off);
                    sb[u] = bf16_bits_to_float(r.s1[grp]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float d[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[n][i] = 0.0f;
                const int k0 = c + u < c1 ? (c + u) * W::kChunk + t * W::kLaneK : K;
#pragma unroll
                for (int j = 0; j < W::kWords; ++j) {
                    const uint32_t wa = a[u][j], wb = b[u][j];
                    const uint32_t a0 = q4_pair(wa), a1 = q4_pair(wa >> 4), a2 = q4_pair(wa >> 8), a3 = q4_pair(wa >> 12);
                    const uint32_t b0 = q4_pair(wb), b1 = q4_pair(wb >> 4), b2 = q4_pair(wb >> 8), b3 = q4_pair(wb >> 12);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 xv = ld_row8<VEC>(x[n], k0 + 8 * j, K);
                        // pairs (k, k + 4): halves of words (0, 2), then (1, 3)
                        const uint32_t x04 = __byte_perm(xv.x, xv.z, 0x5410), x15 = __byte_perm(xv.x, xv.z, 0x7632);
                        const uint32_t x26 = __byte_perm(xv.y, xv.w, 0x5410), x37 = __byte_perm(xv.y, xv.w, 0x7632);
                        mma_bf16(d[n], a0, b0, a1, b1, x04, x15);
                        mma_bf16(d[n], a2, b2, a3, b3, x26, x37);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[n][0] = __fmaf_rn(sa[u], d[n][0], acc[n][0]);
                    acc[n][1] = __fmaf_rn(sa[u], d[n][1], acc[n][1]);
                    acc[n][2] = __fmaf_rn(sb[u], d[n][2], acc[n][2]);
                    acc[n][3] = __fmaf_rn(sb[u], d[n][3], acc[n][3]);
                }
            }
        }
    }
}

}  // namespace simcomm
