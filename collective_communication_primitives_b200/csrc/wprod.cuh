// Products of a weight matrix with few tokens, streamed: the device code that the 4-bit linear and
// the expert layer share.
//
//   D[r][n] = sum_k W[r][k] X[n][k],   16 MT weight rows x 8 NT tokens per warp
//
// Every weight is used once per token, so the job is to keep enough loads in flight and to spend few instructions
// per byte. bf16 weights run at 3 to 5 TB/s on B200, 4-bit weights at 2.5 to 3.1. Those spend 21 (to 8 tokens) or 27 (16)
// instructions on 256 weights, 11 of them to take them apart, but no pipe is full: issue slots are 38 to 49% busy, the
// integer pipe 35 to 48%, the tensor pipe 17 to 29%, with 0.5 to 0.7 warps ready on a scheduler. The warps wait, for
// the results in the chain from a loaded word over its weights and their product to the scaled sum more than for
// memory; twice as many warps wait for each other instead (all measured). Weights are the 16-row
// operand of the matrix instruction (mma.sync m16n8k16) and tokens its 8 columns, so that one token
// wastes no more than 7 columns. A sum over k may be taken in any order as long as both operands use
// the same one, so no weight is ever moved between lanes for the instruction's sake: lane (g, t)
// (g = lane / 4, t = lane % 4) owns rows g and g + 8 of a row tile and whole runs of 8 k's.
//
// Every warp streams its own weights: 64 bytes of each of its rows per stage (32 k's of bf16, 128 of
// 4-bit weights) through a ring of stages in shared memory, copied 16 bytes per lane and row
// (cp.async). The ring costs no registers and no synchronisation between warps, and its copies run on
// from one unit of work into the next. The tokens of a unit are shared by the CTA's warps: a ninth warp
// copies a panel of k's of their rows ahead (one bulk copy per token, completing on an mbarrier), and the
// eight others hand a panel back when they have used it. Rows of a panel are padded so that the lanes'
// 16-byte reads spread over the banks (2-way for 32 consecutive k's per lane, free otherwise). Columns
// without a token hold whatever the panel held before: a column's sums depend on that column alone. A token's values
// may come in two bf16 parts (16 bits of them): the second ones have rows of their own behind the first ones', and
// both go into the same sums.
//
// 4-bit weights (whole numbers set into a float's last bits, as published by Kim, Henry, Fahim and Awadalla, "Who says
// elephants can't run", 2022): word bits 4i..4i+3 hold weight i of eight, value q - 8. (w & 0x000F000F) | 0x43004300
// is the pair (128 + q_0, 128 + q_4) of bf16 values, and subtracting 136 is exact; shifts by 4 give
// the pairs (1,5), (2,6), (3,7); the tokens' words are paired the same way. A chunk's sum is taken
// over the whole numbers q - 8 (bf16 holds them, the products are exact in fp32) and scaled once per
// chunk in fp32, so the weights are never rounded.
//
// Sums are held in fp32 throughout: the matrix instruction's accumulator, then plain adds over the
// warps that share a row tile, in warp order.
#pragma once

#include "common.cuh"
#include "panels.h"

namespace simcomm {

enum WeightKind { W_BF16 = 0, W_Q4X4 = 1, W_Q4X2 = 2, W_Q4X1 = 3 };

template <int WK> struct WTraits {
    static constexpr bool kQ4 = WK != W_BF16;
    static constexpr int kWords = WK == W_Q4X4 ? 4 : WK == W_Q4X2 ? 2 : 1;  // 16-byte token pieces of a lane in a chunk
    static constexpr int kLaneK = 8 * kWords;    // k's of one lane in a chunk
    static constexpr int kChunk = 4 * kLaneK;    // k's of a warp's chunk
    static constexpr int kLaneBytes = kQ4 ? 4 * kWords : 16;  // weight bytes of one lane and row in a chunk
    static constexpr int kChunks = 16 / kLaneBytes;           // chunks of a stage (64 bytes of a row)
    static constexpr int kStageK = kChunks * kChunk;          // k's of a stage
    static constexpr int kPieces = kChunks * kWords;          // 16-byte token pieces of a lane in a stage
};

constexpr int kProdWarps = 8;                       // warps that multiply
constexpr int kProdThreads = (kProdWarps + 1) * 32;  // and one that copies tokens
constexpr int kRing = 4;                            // stages of a warp's weight ring
constexpr int kMaxNT = 4;
template <int WK> constexpr int panel_pad() { return WK == W_Q4X4 ? 32 : WK == W_Q4X2 ? 16 : 64; }  // bytes per row
template <int WK, int NT> constexpr int panel_pitch() { return kPanelK / NT * 2 + panel_pad<WK>(); }
template <int PARTS> constexpr int panel_bytes() { return PARTS * (8 * kPanelK * 2 + 8 * kMaxNT * 64); }
constexpr int kSumTokens = 16;  // tokens whose sums are exchanged at a time where warps share a row tile
template <int MT> constexpr int sums_bytes() { return kProdWarps * MT * 16 * kSumTokens * 4; }
// Shared memory: panels, rings, exchanged sums, mbarriers. PARTS: the most bf16 parts of a token value.
template <int MT, int PARTS> constexpr int product_smem() {
    return kPanels * panel_bytes<PARTS>() + kProdWarps * kRing * MT * 1024 + sums_bytes<MT>() + 3 * kPanels * 8;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a zero addend.
__device__ __forceinline__ void mma_bf16_from0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// 16 bytes from global to shared memory, `bytes` of them read (0: zeros).
__device__ __forceinline__ void cp_async16(uint32_t smem, const void* g, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" :: "r"(smem), "l"(g), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// Eight consecutive bf16 values from element k of a row of K, zero past the end. VEC: K and the row
// are multiples of 16 bytes; otherwise one element at a time.
template <bool VEC> __device__ __forceinline__ uint4 ld_row8(const uint16_t* row, int k, int K) {
    if (!row || k >= K) return make_uint4(0u, 0u, 0u, 0u);
    if constexpr (VEC) {
        return *reinterpret_cast<const uint4*>(row + k);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0u, hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0u;
            w[i] = lo | hi << 16;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Eight tokens' values (0..7) as the pairs (0,4) (1,5) (2,6) (3,7), which is how a word's 4-bit weights come apart.
__device__ __forceinline__ uint4 paired(uint4 v) {
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                      __byte_perm(v.y, v.w, 0x7632));
}

// Whether a panel holds its tokens in pairs: the copying warp then makes them once for all, else every warp as it
// reads. With up to 8 tokens a panel is long and the copying warp has the time: 48 and 45 us at 65536 x 4096 with one
// token on B200, every warp and once. With more it has not: 117 and 124 at 131072 x 4096 with 16, 49 and 60 at 16384 x
// 4096 with 64.
template <int WK, int NT> constexpr bool panel_pairs() { return WTraits<WK>::kQ4 && NT == 1; }

// The constants of the 4-bit form, held in registers: a logic instruction takes one immediate, and the
// mask and the bias go into one.
struct Q4Consts { uint32_t mask, bias; };
__device__ __forceinline__ Q4Consts q4_consts() {
    Q4Consts c;
    asm volatile("mov.u32 %0, 0x000F000F; mov.u32 %1, 0x43004300;" : "=r"(c.mask), "=r"(c.bias));
    return c;
}
// Two bf16 values q - 8 of the nibble pair (i, i + 4) of a word shifted right by 4 i.
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, const Q4Consts& c) {
    uint32_t biased, r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(biased) : "r"(w), "r"(c.mask), "r"(c.bias));  // (w & mask) | bias
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(biased), "r"(0x43084308u));
    return r;
}

// The place of 16-byte piece p of row (m, i, g) in a ring stage. Rows lie 64 bytes apart; the pieces of a
// row are permuted by g so that reads of 4, 8 and 16 bytes per lane all spread over the banks.
__device__ __forceinline__ uint32_t ring_at(int m, int i, int g, int p) {
    const int swz = ((g >> 1) & 1) << 1 | g >> 2;
    return uint32_t(((m * 2 + i) * 8 + g) * 64 + ((p ^ swz) << 4));
}

// Starts the copy of one stage of the warp's weights (64 bytes of each row) into the ring.
template <int WK, bool VEC, int MT>
__device__ __forceinline__ void fetch_stage(uint32_t ring, const char* const (&w)[MT][2], int stage, int K, int g, int t) {
    using W = WTraits<WK>;
    const int k = stage * W::kStageK + t * (W::kStageK / 4);  // first k of the lane's 16 bytes
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t to = ring + ring_at(m, i, g, t);
            if constexpr (VEC) {
                cp_async16(to, w[m][i] + (k < K ? size_t(stage) * 64 + t * 16 : 0), k < K ? 16u : 0u);
            } else {
                const uint4 v = ld_row8<false>(reinterpret_cast<const uint16_t*>(w[m][i]), k, K);
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                             : "memory");
            }
        }
}

// The scales of a stage's rows, one per chunk, Lane t of a quad loads those of rows (2 q + t / 2,
// t % 2) (with one row tile: (0, t % 2)), a stage ahead (a row's scales lie together, so that most of these loads hit L1), and they
// are exchanged when they are used.
template <int WK, int MT> struct StageScales { uint16_t v[(MT + 1) / 2][WTraits<WK>::kChunks]; };

template <int WK, int MT>
__device__ __forceinline__ void load_scales(StageScales<WK, MT>& sc, const uint16_t* const (&s)[(MT + 1) / 2], int stage, int groups, int shift) {
    using W = WTraits<WK>;
#pragma unroll
    for (int u = 0; u < W::kChunks; ++u) {
        const int grp = min((stage * W::kChunks + u) >> shift, groups - 1);
#pragma unroll
        for (int q = 0; q < (MT + 1) / 2; ++q) sc.v[q][u] = __ldg(s[q] + grp);
    }
}

template <int BYTES> __device__ __forceinline__ void lds(uint32_t (&v)[4], const unsigned char* at) {
    if constexpr (BYTES == 16) {
        const uint4 q = *reinterpret_cast<const uint4*>(at);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else if constexpr (BYTES == 8) {
        const uint2 q = *reinterpret_cast<const uint2*>(at);
        v[0] = q.x; v[1] = q.y;
    } else {
        v[0] = *reinterpret_cast<const uint32_t*>(at);
    }
}

// acc += one stage, whose tokens' k's start at `tok` of the panel (at this lane's token and first k).
template <int WK, int MT, int NT, int PARTS>
__device__ __forceinline__ void use_stage(float (&acc)[MT][NT][4], const unsigned char* ring, const StageScales<WK, MT>& sc,
                                          const unsigned char* tok, int g, int t, const Q4Consts& qc) {
    using W = WTraits<WK>;
    constexpr int kPitch = panel_pitch<WK, NT>();
    auto token8 = [&](int part, int n, int u, int j) {  // run j of 8 k's of chunk u
        const uint4 v = *reinterpret_cast<const uint4*>(tok + (part * NT + n) * 8 * kPitch + u * W::kChunk * 2 + j * 16);
        return W::kQ4 && !panel_pairs<WK, NT>() ? paired(v) : v;
    };
    if constexpr (!W::kQ4) {
        uint4 x[PARTS][NT];
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
#pragma unroll
            for (int n = 0; n < NT; ++n) x[q][n] = token8(q, n, 0, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            uint32_t a[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) lds<16>(a[i], ring + ring_at(m, i, g, t));
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_bf16(acc[m][n], a[0][0], a[1][0], a[0][1], a[1][1], x[q][n].x, x[q][n].y);
                    mma_bf16(acc[m][n], a[0][2], a[1][2], a[0][3], a[1][3], x[q][n].z, x[q][n].w);
                }
        }
    } else {
        // a chunk's tokens are held for all row tiles, unless they are too many registers
        constexpr bool kHold = W::kWords * NT * PARTS <= 8;
#pragma unroll
        for (int u = 0; u < W::kChunks; ++u) {
            uint4 x[kHold ? W::kWords : 1][PARTS][NT];
            if constexpr (kHold) {
#pragma unroll
                for (int j = 0; j < W::kWords; ++j)
#pragma unroll
                    for (int q = 0; q < PARTS; ++q)
#pragma unroll
                        for (int n = 0; n < NT; ++n) x[j][q][n] = token8(q, n, u, j);
            }
            const int byte = (4 * u + t) * W::kLaneBytes;  // of the row's 64
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t w[2][4];
                float d[NT][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) lds<W::kLaneBytes>(w[i], ring + ring_at(m, i, g, byte >> 4) + (byte & 15));
#pragma unroll
                for (int j = 0; j < W::kWords; ++j) {
                    if constexpr (!kHold) {
#pragma unroll
                        for (int q = 0; q < PARTS; ++q)
#pragma unroll
                            for (int n = 0; n < NT; ++n) x[0][q][n] = token8(q, n, u, j);
                    }
                    const uint32_t wa = w[0][j], wb = w[1][j];
                    const uint32_t a0 = q4_pair(wa, qc), a1 = q4_pair(wa >> 4, qc), a2 = q4_pair(wa >> 8, qc), a3 = q4_pair(wa >> 12, qc);
                    const uint32_t b0 = q4_pair(wb, qc), b1 = q4_pair(wb >> 4, qc), b2 = q4_pair(wb >> 8, qc), b3 = q4_pair(wb >> 12, qc);
#pragma unroll
                    for (int q = 0; q < PARTS; ++q)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4 v = x[kHold ? j : 0][q][n];
                            if (j == 0 && q == 0) mma_bf16_from0(d[n], a0, b0, a1, b1, v.x, v.y);
                            else mma_bf16(d[n], a0, b0, a1, b1, v.x, v.y);
                            mma_bf16(d[n], a2, b2, a3, b3, v.z, v.w);
                        }
                }
                const int from = (threadIdx.x & 28) + 2 * (m % 2);  // the quad's lane that holds row (m, 0)
                const float sa = bf16_bits_to_float(__shfl_sync(0xffffffffu, uint32_t(sc.v[m / 2][u]), from));
                const float sb = bf16_bits_to_float(__shfl_sync(0xffffffffu, uint32_t(sc.v[m / 2][u]), from + 1));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[m][n][0] = __fmaf_rn(sa, d[n][0], acc[m][n][0]);
                    acc[m][n][1] = __fmaf_rn(sa, d[n][1], acc[m][n][1]);
                    acc[m][n][2] = __fmaf_rn(sb, d[n][2], acc[m][n][2]);
                    acc[m][n][3] = __fmaf_rn(sb, d[n][3], acc[m][n][3]);
                }
            }
        }
    }
}

// ---- the work of a CTA -----------------------------------------------------------------------------
//
// A Job describes a sequence of units; the CTA takes units first, first + step, ... A unit is a block of row
// tiles against up to 8 NT tokens, summed over `segments` rows of K each (the ranks of a sum over ranks).
// Some warps (1, 2, 4 or 8) share each row tile, the stages of a segment dealt to them in turn. A Job has
//   static kWK, kVecW, kVecX, kMT;   int K, segments, chunk_shift
//   int split_shift(unit)                log2 of the warps that share a row tile
//   void rows(unit, seg, tile, g, w)     the lane's weight rows of the CTA's tile-th row tile group
//   void scales(unit, seg, tile, g, t, s)
//   const uint16_t* token(unit, seg, n)  row of the n-th token, null for none
//   ptrdiff_t part                       elements from a row to that of its values' second parts

// Most warps that can share a row tile: every panel has a stage for each.
template <int WK, int NT> constexpr int max_splits() {
    return kPanelK / NT / WTraits<WK>::kStageK < kProdWarps ? kPanelK / NT / WTraits<WK>::kStageK : kProdWarps;
}

struct ProductSmem {
    unsigned char* base;
    int panel;        // bytes of a buffer
    int rings, sums;  // bytes from base
    uint64_t* full;   // [kPanels]: the panel's tokens are in
    uint64_t* landed; // [kPanels]: they are in, but not yet in pairs (panel_pairs)
    uint64_t* empty;  // [kPanels]: every multiplying warp has used it
};
template <int MT, int PARTS> __device__ __forceinline__ ProductSmem product_layout(unsigned char* smem) {
    ProductSmem s;
    s.base = smem;
    s.panel = panel_bytes<PARTS>();
    s.rings = kPanels * s.panel;
    s.sums = s.rings + kProdWarps * kRing * MT * 1024;
    s.full = reinterpret_cast<uint64_t*>(smem + s.sums + sums_bytes<MT>());
    s.empty = s.full + kPanels;
    s.landed = s.empty + kPanels;
    return s;
}
// By one thread, before a __syncthreads.
__device__ __forceinline__ void init_panels(const ProductSmem& s) {
    for (int i = 0; i < kPanels; ++i) {
        mbar_init(&s.full[i], 1);
        mbar_init(&s.landed[i], 1);
        mbar_init(&s.empty[i], kProdWarps);
    }
    fence_barrier_init();
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_u32(bar)) : "memory");
}

constexpr uint64_t kLandNs = 1000000000ull;  // longest wait for copies in flight before a CTA may leave

// The copying warp's side of a unit. False after a wait that ran out.
template <int NT, int PARTS, typename Job>
__device__ __forceinline__ bool copy_tokens(const Job& job, const Ctl& ctl, uint64_t timeout_ns, const ProductSmem& s,
                                            PanelCount& pc, int unit) {
    using W = WTraits<Job::kWK>;
    constexpr int kPitch = panel_pitch<Job::kWK, NT>(), kSpan = kPanelK / NT, kPart = 8 * NT * kPitch;
    constexpr bool kPairs = panel_pairs<Job::kWK, NT>();
    const int lane = threadIdx.x & 31;
    for (int seg = 0; seg < job.segments; ++seg) {
        const uint16_t* row = lane < 8 * NT ? job.token(unit, seg, lane) : nullptr;
        const uint32_t rows = __popc(__ballot_sync(0xffffffffu, row != nullptr));
        for (int k0 = 0; k0 < job.K; k0 += kSpan, ++pc.n) {
            const int buf = pc.buf(), n = min(kSpan, job.K - k0);
            const int padded = (n + W::kStageK - 1) / W::kStageK * W::kStageK;  // a stage is read whole
            if (!mbar_wait_warp(ctl, &s.empty[buf], pc.parity() ^ 1u, timeout_ns)) return false;
            unsigned char* panel = s.base + buf * s.panel;
            if constexpr (Job::kVecX) {
                unsigned char* to = panel + lane * kPitch;
                if (padded > n && row)  // zeros past the row's end
                    for (int q = 0; q < PARTS; ++q)
                        for (int k = n; k < padded; k += 8)
                            *reinterpret_cast<uint4*>(to + q * kPart + k * 2) = make_uint4(0u, 0u, 0u, 0u);
                // This warp's ordinary writes to the buffer come before the copies that follow: zeros, those of the
                // panel that it held before (of any length), and that panel's pairs (of a unit that makes them, which
                // this one need not be).
                fence_proxy_async_smem();
                __syncwarp();
                uint64_t* in = kPairs ? &s.landed[buf] : &s.full[buf];
                if (lane == 0) mbar_arrive_expect_tx(in, rows * uint32_t(n) * (2u * PARTS));
                __syncwarp();
                if (row)
#pragma unroll
                    for (int q = 0; q < PARTS; ++q)
                        bulk_g2s(to + q * kPart, row + q * job.part + k0, uint32_t(n) * 2u, in);
                if constexpr (kPairs) {  // put into pairs where they lie
                    if (!mbar_wait_warp(ctl, in, pc.landed_parity(), timeout_ns)) {
                        mbar_wait_warp(ctl, in, pc.landed_parity(), kLandNs);
                        return false;
                    }
                    pc.used_landed();
                    constexpr int kPieces = kSpan / 256, kRows = 8 / kPieces;  // of a lane and row; rows at a time
                    for (int part = 0; part < PARTS; ++part) {
                        unsigned char* rows_of = panel + part * kPart;
                        for (uint32_t i = 0; i < rows; i += kRows) {
                            uint4 v[kRows][kPieces];
#pragma unroll
                            for (int h = 0; h < kRows; ++h)
#pragma unroll
                                for (int q = 0; q < kPieces; ++q)
                                    if (i + h < rows) v[h][q] = *reinterpret_cast<const uint4*>(rows_of + (i + h) * kPitch + (q * 32 + lane) * 16);
#pragma unroll
                            for (int h = 0; h < kRows; ++h)
#pragma unroll
                                for (int q = 0; q < kPieces; ++q)
                                    if (i + h < rows) *reinterpret_cast<uint4*>(rows_of + (i + h) * kPitch + (q * 32 + lane) * 16) = paired(v[h][q]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.full[buf]);
                }
            } else {  // by loads and stores, the pieces of two rows in flight
                constexpr int kPieces = kSpan / 256;  // of a lane and row
                const uint64_t at = reinterpret_cast<uint64_t>(row);
                for (int part = 0; part < PARTS; ++part)
                    for (uint32_t i = 0; i < rows; i += 2) {
                        uint4 v[2][kPieces];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const auto* from = reinterpret_cast<const uint16_t*>(__shfl_sync(0xffffffffu, at, int(i) + h));
#pragma unroll
                            for (int q = 0; q < kPieces; ++q)
                                v[h][q] = ld_row8<Job::kVecX>(i + h < rows ? from + part * job.part : nullptr, k0 + (q * 32 + lane) * 8, job.K);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int q = 0; q < kPieces; ++q)
                                if (i + h < rows && (q * 32 + lane) * 8 < padded)
                                    *reinterpret_cast<uint4*>(panel + part * kPart + (i + h) * kPitch + (q * 32 + lane) * 16) =
                                        kPairs ? paired(v[h][q]) : v[h][q];
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.full[buf]);
            }
        }
    }
    return true;
}

// The copying warp's last step, after its units or a wait that ran out: its copies are in before the CTA can leave, for
// they write the CTA's shared memory. (The multiplying warps wait for them too, unless their waits run out.)
__device__ __forceinline__ void land_panels(const Ctl& ctl, const ProductSmem& s, PanelCount pc) {
    for (int i = 0; i < kPanels && pc.n > 0; ++i) {
        --pc.n;
        mbar_wait_warp(ctl, &s.full[pc.buf()], pc.parity(), kLandNs);
    }
}

// Where a multiplying warp's copies have got to: a stage of a segment of a unit.
template <int MT> struct Ahead {
    const char* w[MT][2];
    int unit, seg, next, slot, splits;
};

template <typename Job> struct Multiplier {
    using W = WTraits<Job::kWK>;
    static constexpr int MT = Job::kMT;
    const Job& job;
    const ProductSmem& s;
    int units, step;           // of the CTA's sequence: units below `units`, every `step`-th
    int warp, lane, g, t, stages;
    uint32_t ring;
    int slot = 0;
    bool live = true;          // false after a wait that ran out: the warp's sums are 0, and it only meets the others
    Ahead<MT> ahead;
    Q4Consts qc;

    __device__ __forceinline__ Multiplier(const Job& j, const ProductSmem& sm, int first, int units_, int step_)
        : job(j), s(sm), units(units_), step(step_) {
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        g = lane >> 2;
        t = lane & 3;
        stages = (job.K + W::kStageK - 1) / W::kStageK;
        ring = smem_u32(s.base) + s.rings + warp * (kRing * MT * 1024);
        qc = q4_consts();
        ahead.unit = first;
        ahead.seg = 0;
        ahead.slot = 0;
        ahead.next = ahead.splits = 1;
        if (first < units) start_rows();
        __syncwarp();  // an earlier use of the ring by this warp is over
#pragma unroll
        for (int i = 0; i < kRing - 1; ++i) fetch();
    }

    // Turns the copies to their segment's rows.
    __device__ __forceinline__ void start_rows() {
        const int shift = job.split_shift(ahead.unit);
        ahead.splits = 1 << shift;
        ahead.next = warp & (ahead.splits - 1);
        job.rows(ahead.unit, ahead.seg, warp >> shift, g, ahead.w);
    }

    // Starts the next copy of the sequence; past its end an empty group keeps the count of groups in step.
    __device__ __forceinline__ void fetch() {
        while (ahead.next >= stages && ahead.unit < units) {
            if (++ahead.seg == job.segments) {
                ahead.seg = 0;
                ahead.unit += step;
            }
            if (ahead.unit < units) start_rows();
        }
        if (ahead.unit < units) {
            fetch_stage<Job::kWK, Job::kVecW, MT>(ring + ahead.slot * (MT * 1024), ahead.w, ahead.next, job.K, g, t);
            ahead.next += ahead.splits;
            ahead.slot = ahead.slot + 1 == kRing ? 0 : ahead.slot + 1;
        }
        cp_async_commit();
    }

    // The warp's sums of a unit over its share of the stages (0 where the warp is not live). Every warp of the CTA goes
    // through all units, since warps that share a row tile meet at a barrier.
    template <int NT, int PARTS>
    __device__ __forceinline__ void unit(const Ctl& ctl, uint64_t timeout_ns, PanelCount& pc, int u, float (&acc)[MT][NT][4]) {
        constexpr int kPitch = panel_pitch<Job::kWK, NT>(), kPanelStages = kPanelK / NT / W::kStageK;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
        if (!live) return;
        const int shift = job.split_shift(u), splits = 1 << shift, tile = warp >> shift, split = warp & (splits - 1);
        const int groups = (((job.K + W::kChunk - 1) / W::kChunk - 1) >> job.chunk_shift) + 1;
        for (int seg = 0; seg < job.segments; ++seg) {
            const uint16_t* sp[(MT + 1) / 2];
            StageScales<Job::kWK, MT> next;
            if constexpr (W::kQ4) {
                job.scales(u, seg, tile, g, t, sp);
                load_scales<Job::kWK, MT>(next, sp, split, groups, job.chunk_shift);
            }
            int st = split;
            for (int p0 = 0; p0 < stages; p0 += kPanelStages, ++pc.n) {
                const int buf = pc.buf(), end = min(p0 + kPanelStages, stages);
                if (!mbar_wait_warp(ctl, &s.full[buf], pc.parity(), timeout_ns)) {
                    live = false;
                    return;
                }
                const unsigned char* tok = s.base + buf * s.panel + g * kPitch + t * W::kLaneK * 2;
                for (; st < end; st += splits) {
                    const StageScales<Job::kWK, MT> sc = next;
                    if constexpr (W::kQ4) load_scales<Job::kWK, MT>(next, sp, st + splits, groups, job.chunk_shift);
                    cp_async_wait<kRing - 2>();
                    __syncwarp();  // the stage is in for every lane, and the slot refilled next has been read
                    fetch();
                    use_stage<Job::kWK, MT, NT, PARTS>(acc, s.base + s.rings + (warp * kRing + slot) * (MT * 1024), sc,
                                                tok + (st - p0) * (W::kStageK * 2), g, t, qc);
                    slot = slot + 1 == kRing ? 0 : slot + 1;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.empty[buf]);
            }
        }
    }

    // Host-side fault injection: the warp falls silent, as after a wait that ran out.
    __device__ __forceinline__ void give_up() { live = false; }

    // After the last unit: waits for the warp's copies in flight (none after a whole sequence but empty groups), and
    // reports sums that are missing, in case nobody had to wait for this warp.
    __device__ __forceinline__ void drain(const Ctl& ctl) {
        cp_async_wait<0>();
        if (!live && lane == 0) raise_status(ctl, COLL_ERR_TIMEOUT);
    }
};

__device__ __forceinline__ void sync_multipliers() { asm volatile("bar.sync 1, %0;" :: "n"(kProdWarps * 32) : "memory"); }

// Calls out(row tile group, row, token, value) for every finished sum of the CTA's unit: row of the 16 MT of a
// group of row tiles, token below 8 NT. With one warp per group straight from its registers; otherwise the
// warps' sums meet in shared memory and are added in warp order. PAIR: value2 is the sum 8 rows below, for
// rows with bit 3 clear (the others are not called).
template <bool PAIR, int MT, int NT, typename Out>
__device__ __forceinline__ void finish_unit(const ProductSmem& s, int splits, const float (&acc)[MT][NT][4], Out out) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (splits == 1) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = n * 8 + 2 * t + j;
                    if constexpr (PAIR) {
                        out(warp, m * 16 + g, c, acc[m][n][j], acc[m][n][2 + j]);
                    } else {
                        out(warp, m * 16 + g, c, acc[m][n][j], 0.0f);
                        out(warp, m * 16 + 8 + g, c, acc[m][n][2 + j], 0.0f);
                    }
                }
        return;
    }
    float* sums = reinterpret_cast<float*>(s.base + s.sums);
    constexpr int NB = NT < kSumTokens / 8 ? NT : kSumTokens / 8;  // token tiles at a time
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += NB) {
        sync_multipliers();  // the last exchange has been read
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[(((warp * MT + m) * NB + n) * 4 + i) * 32 + lane] = acc[m][n0 + n][i];
        sync_multipliers();
        constexpr int kPerGroup = MT * NB * 2 * 32 * (PAIR ? 1 : 2);  // sums of a group of row tiles
        const int all = kProdWarps / splits * kPerGroup;
        for (int e = threadIdx.x; e < all; e += kProdWarps * 32) {
            const int q = e / kPerGroup, rest = e % kPerGroup, ln = rest % 32, reg = rest / 32;
            const int j = reg % 2, half = PAIR ? 0 : reg / 2 % 2, n = reg / (PAIR ? 2 : 4) % NB, m = reg / (PAIR ? 2 : 4) / NB;
            const float* at = sums + (((q * splits * MT + m) * NB + n) * 4 + half * 2 + j) * 32 + ln;
            float v = 0.0f, v2 = 0.0f;
            for (int w = 0; w < splits; ++w) {
                v += at[w * (MT * NB * 128)];
                if (PAIR) v2 += at[w * (MT * NB * 128) + 64];
            }
            out(q, m * 16 + half * 8 + ln / 4, (n0 + n) * 8 + ln % 4 * 2 + j, v, v2);
        }
    }
}

}  // namespace simcomm
