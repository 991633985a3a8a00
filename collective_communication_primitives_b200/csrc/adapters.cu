// Low-rank adapters of many requests beside a shared projection.
//
//   u[t] = A_e x[t]  (summed over the ranks in the row-parallel form),  out[t] = base[t] + scale[e] B_e u[t],  e = adapter[t]
//
// Two kernels: k_adapter_down forms u, k_adapter_up adds B u to the base. Tokens are taken in groups of 8 or 32 that follow each
// other, and a group once for each adapter that occurs in it, with the other adapters' tokens masked out: a decode step's
// tokens, each with an adapter of its own, stream every matrix once, a prompt's tokens share one. The matrix instruction
// (mma.sync m16n8k16) has the matrices' rows as its 16-row operand and tokens as its 8 columns, as in the products with
// 4-bit weights: a few tokens fill 8 columns and would leave most of a 128-row tcgen05 tile empty, and a rank of 16 is one
// step of k. Its operands come from memory in the order they lie in: within a step the k's are dealt to the lanes so that a lane's
// are neighbours (both operands alike, so the sum is the same), which makes them 16-byte (down) and 8-byte (up) loads
// without shared memory, and the rows of B so that a lane's four results of a token are neighbours.
//
// u is fp32, its parts over k joined in order by the second kernel, which splits it into bf16 numbers that add up to it, since B u
// would otherwise carry a rounding of 2^-9: two where out is bf16 (what is lost is 2^-16 of it or less), three where it is fp32 (2^-24).
// The second kernel starts while the first ends and
// waits for it only where it needs u. Bound by the bytes of the tokens, outputs and met adapters; in a decode step by the
// latency of loads that wait for each other (a token's adapter, its matrices, u, the base). Measured on B200, replayed in a
// graph: 32 tokens of 64 adapters of rank 16, row-parallel over 8 ranks, 14 us (13 MB, 0.9 TB/s); 4099 tokens of 8
// adapters of rank 64, 4096 x 4096, column-parallel, 48.5 us, of which the first kernel has 22 and the second 33 beside its
// early start (105 MB, 2.2 TB/s; the matrices come from L2 once for every 32 tokens, another 134 MB). There the
// tensor pipe is 29% busy and 41% of the issue slots are used: two CTAs of 128 registers a thread leave a scheduler four warps.
#include <algorithm>

#include "common.cuh"
#include "wprod.cuh"

namespace simcomm {

constexpr int kAdThreads = 256;
constexpr int kAdWarps = kAdThreads / 32;
constexpr int kAdChunk = 32;   // k's of one step of k_adapter_down: two matrix instructions
constexpr int kAdChain = 4096; // k's that are summed by matrix instructions alone
constexpr int kAdParts = 16;   // parts of the sum over k at most

// The group's tokens by adapter: each lane's own adapter (-1: none), the lanes with the same one, and a bit for each first of
// them. The same for every warp.
struct Crews {
    int mine;
    uint32_t same, firsts;
};
__device__ __forceinline__ Crews crews_of(const AdapterArgs& a, size_t t0, int group, bool none_too) {
    const int lane = threadIdx.x & 31;
    const bool here = lane < group && t0 + lane < a.T;
    int e = here ? a.adapter[t0 + lane] : -2;
    if (here && (e < -1 || e >= a.adapters)) {
        raise_status(a.ctl, COLL_ERR_INVALID_ARG);
        e = -1;
    }
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const bool counts = e >= 0 || (e == -1 && none_too);
    return Crews{e, same, __ballot_sync(0xffffffffu, counts && (same & ((1u << lane) - 1u)) == 0u)};
}
__device__ __forceinline__ int rank_of(const AdapterArgs& a, int e) {
    if (e < 0) return 0;
    const int r = a.rank ? a.rank[e] : a.R;
    if (r >= 0 && r <= a.R) return r;
    raise_status(a.ctl, COLL_ERR_INVALID_ARG);
    return 0;
}

// Eight bf16 from k on, zeros past the row's end.
template <bool VEC> __device__ __forceinline__ uint4 load8(const uint16_t* row, size_t k, size_t K) {
    if constexpr (VEC) {
        return k < K ? __ldg(reinterpret_cast<const uint4*>(row + k)) : make_uint4(0, 0, 0, 0);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0u, hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0u;
            w[i] = lo | (hi << 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// NT: tokens of a group in eights. MT: tiles of 16 rows of A that a warp takes at once; the warps share the steps of k, so that a
// CTA loads tokens and rows once (with the tiles on different warps 4099 tokens at rank 64 took 66 us, the tokens loaded four times).
// LONG: a part has more than kAdChain k's, and the warps' sums are added to u after as many of them.
template <int NT, int MT, bool VEC, bool LONG> __global__ void __launch_bounds__(kAdThreads, NT * MT > 4 ? 1 : 2)
k_adapter_down(const __grid_constant__ AdapterArgs a, int slots) {
    constexpr int kAhead = 2 * MT + NT > 8 ? 2 : 4;           // steps whose loads are in flight
    constexpr int kPart = MT * NT > 8 ? 8 / MT : NT;          // eights of tokens whose sums the warps exchange at a time
    __shared__ float s_sum[kAdWarps][16 * MT * 8 * kPart];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool failed = status_failed(a.ctl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t b = blockIdx.x / a.splits, groups = gridDim.x / a.splits / slots;
    const int split = int(blockIdx.x % a.splits), sub = slots - 1 - int(b / groups);  // CTAs that may have nothing to do come first
    const size_t t0 = size_t(b % groups) * (8 * NT);
    const uint32_t steps = uint32_t((a.K + kAdChunk - 1) / kAdChunk), all = steps * a.segments;
    const uint32_t s0 = uint32_t(uint64_t(all) * split / a.splits), s1 = uint32_t(uint64_t(all) * (split + 1) / a.splits);
    const Crews crews = crews_of(a, t0, 8 * NT, false);
    if (__popc(crews.firsts) <= sub) return;
    if (__syncthreads_or(failed)) return;
    uint32_t todo = crews.firsts;
    for (int crew = 0; todo; ++crew) {
        const int slot = __ffs(todo) - 1;
        todo &= todo - 1;
        if (crew % slots != sub) continue;
        const int adapter = __shfl_sync(0xffffffffu, crews.mine, slot);
        const uint32_t tokens = __shfl_sync(0xffffffffu, crews.same, slot);
        const int R = rank_of(a, adapter), tiles = (R + 15) / 16;
        for (int tile0 = 0; tile0 < tiles; tile0 += MT) {
            uint32_t b1 = 0;
            for (uint32_t b0 = s0; b0 < s1; b0 = b1) {
                b1 = LONG ? min(b0 + kAdChain / kAdChunk, s1) : s1;
                float acc[MT][NT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.0f;
                }
                size_t at_row[MT][2];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i)  // rows past the adapter's: its last one
                        at_row[m][i] = (size_t(adapter) * a.R + min((tile0 + m) * 16 + g + 8 * i, R - 1)) * a.K;
                for (uint32_t s = b0 + warp; s < b1; s += kAdWarps * kAhead) {
                    uint4 w[kAhead][MT][2], x[kAhead][NT];
#pragma unroll
                    for (int q = 0; q < kAhead; ++q) {
                        const uint32_t at = s + q * kAdWarps;
                        const uint32_t seg = at < b1 && a.segments > 1 ? at / steps : 0u;
                        const size_t k = at < b1 ? size_t(at - seg * steps) * kAdChunk + c * 8 : a.K;
                        const uint16_t* matrix = a.a[a.rank0 + seg];
                        const uint16_t* v = a.x[a.rank0 + seg];
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                w[q][m][i] = tile0 + m < tiles ? load8<VEC>(matrix + at_row[m][i], k, a.K) : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            x[q][n] = (tokens >> (8 * n + g)) & 1u ? load8<VEC>(v + (t0 + 8 * n + g) * a.K, k, a.K) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int q = 0; q < kAhead; ++q)
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const uint4 &w0 = w[q][m][0], &w1 = w[q][m][1];
                                mma_bf16(acc[m][n], w0.x, w1.x, w0.y, w1.y, x[q][n].x, x[q][n].y);
                                mma_bf16(acc[m][n], w0.z, w1.z, w0.w, w1.w, x[q][n].z, x[q][n].w);
                            }
                }
                // a lane's sums: row g or g + 8 of a tile, tokens 2c and 2c + 1 of eight n
#pragma unroll
                for (int n0 = 0; n0 < NT; n0 += kPart) {
                    if (n0 > 0 || tile0 > 0 || (LONG && b0 > s0)) __syncthreads();
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int n = 0; n < kPart; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                s_sum[warp][(8 * n + 2 * c + (i & 1)) * (16 * MT) + m * 16 + g + 8 * (i >> 1)] = acc[m][n0 + n][i];
                    __syncthreads();
                    for (int i = threadIdx.x; i < 16 * MT * 8 * kPart; i += kAdThreads) {
                        const int row = tile0 * 16 + i % (16 * MT), t = 8 * n0 + i / (16 * MT);
                        if (row >= R || !((tokens >> t) & 1u)) continue;
                        float v = s_sum[0][i];
#pragma unroll
                        for (int d = 1; d < kAdWarps; ++d) v += s_sum[d][i];
                        float* u = a.u + (size_t(split) * a.T + t0 + t) * a.Rp + row;
                        *u = LONG && b0 > s0 ? *u + v : v;  // an element is one thread's every time
                    }
                }
            }
        }
        __syncthreads();
    }
}

// The same for groups of 32 tokens whose rows are whole 16-byte units: tokens and rows of A go through a ring of stages in
// shared memory (cp.async), 128 k's of each, of which a warp takes 16. In registers 4099 tokens at rank 64 took 40 us: what is
// loaded ahead there is at most what the registers hold, two steps of a warp.
constexpr int kTileK = 128;                    // k's of a stage
constexpr int kTilePitch = kTileK * 2 + 16;    // bytes of a row of a stage: the 8 rows of a matrix lie on different banks
constexpr int kTileStages = 4;
template <int MT> constexpr int tile_bytes() { return (16 * MT + 32) * kTilePitch; }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t smem) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem) : "memory");
}

template <int MT, bool LONG> __global__ void __launch_bounds__(kAdThreads, 2) k_adapter_down_tiles(const __grid_constant__ AdapterArgs a, int slots) {
    constexpr int NT = 4;
    static_assert(kAdWarps * 16 == kTileK, "a warp has 16 k's of a stage");
    static_assert(kAdWarps * 16 * MT * 8 * NT * 4 <= kTileStages * tile_bytes<MT>(), "the warps' sums lie where the stages did");
    extern __shared__ __align__(128) unsigned char s_tile[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool failed = status_failed(a.ctl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t b = blockIdx.x / a.splits, groups = gridDim.x / a.splits / slots;
    const int split = int(blockIdx.x % a.splits), sub = slots - 1 - int(b / groups);  // CTAs that may have nothing to do come first
    const size_t t0 = size_t(b % groups) * (8 * NT);
    const uint32_t per = uint32_t((a.K + kTileK - 1) / kTileK), all = per * a.segments;  // stages of a rank's columns, in all
    const uint32_t s0 = uint32_t(uint64_t(all) * split / a.splits), s1 = uint32_t(uint64_t(all) * (split + 1) / a.splits);
    const Crews crews = crews_of(a, t0, 8 * NT, false);
    if (__popc(crews.firsts) <= sub) return;
    if (__syncthreads_or(failed)) return;
    const uint32_t base = smem_u32(s_tile);
    float* const sums = reinterpret_cast<float*>(s_tile);
    uint32_t todo = crews.firsts;
    for (int crew = 0; todo; ++crew) {
        const int slot = __ffs(todo) - 1;
        todo &= todo - 1;
        if (crew % slots != sub) continue;
        const int adapter = __shfl_sync(0xffffffffu, crews.mine, slot);
        const uint32_t tokens = __shfl_sync(0xffffffffu, crews.same, slot);
        const int R = rank_of(a, adapter), tiles = (R + 15) / 16;
        for (int tile0 = 0; tile0 < tiles; tile0 += MT) {
            // a thread copies the same 8 k's of every 16th row
            const int piece = threadIdx.x & 15, row0 = threadIdx.x >> 4;
            size_t at[MT + 2];
            bool some[MT + 2];
#pragma unroll
            for (int i = 0; i < MT + 2; ++i) {
                const int t = 16 * (i - MT) + row0;  // a token
                some[i] = i < MT ? tile0 + i < tiles : (tokens >> (t & 31)) & 1u;
                at[i] = i < MT ? (size_t(adapter) * a.R + min((tile0 + i) * 16 + row0, R - 1)) * a.K
                               : (t0 + (some[i] ? t : 0)) * a.K;
            }
            uint32_t b1 = 0;
            for (uint32_t b0 = s0; b0 < s1; b0 = b1) {
                b1 = LONG ? min(b0 + kAdChain / kTileK, s1) : s1;
                auto copy = [&](uint32_t s) {
                    if (s < b1) {
                        const uint32_t seg = a.segments > 1 ? s / per : 0u;
                        const size_t k = size_t(s - seg * per) * kTileK + piece * 8;
                        const uint16_t* m = a.a[a.rank0 + seg];
                        const uint16_t* x = a.x[a.rank0 + seg];
                        const uint32_t to = base + (s % kTileStages) * tile_bytes<MT>() + row0 * kTilePitch + piece * 16;
                        const bool in = k < a.K;
#pragma unroll
                        for (int i = 0; i < MT + 2; ++i)
                            cp_async16(to + i * 16 * kTilePitch, (i < MT ? m : x) + (in ? at[i] + k : 0), in && some[i] ? 16u : 0u);
                    }
                    cp_async_commit();
                };
                float acc[MT][NT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.0f;
#pragma unroll
                for (int q = 0; q < kTileStages - 1; ++q) copy(b0 + q);
                for (uint32_t s = b0; s < b1; ++s) {
                    asm volatile("cp.async.wait_group %0;" :: "n"(kTileStages - 2) : "memory");
                    __syncthreads();  // the stage is in, and the one before it is used up
                    copy(s + kTileStages - 1);
                    const uint32_t from = base + (s % kTileStages) * tile_bytes<MT>() + warp * 32;
                    uint32_t x[NT / 2][4];
#pragma unroll
                    for (int n = 0; n < NT / 2; ++n)
                        ldmatrix4(x[n], from + (16 * MT + 16 * n + (lane >> 4) * 8 + (lane & 7)) * kTilePitch + ((lane >> 3) & 1) * 16);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        uint32_t w[4];
                        ldmatrix4(w, from + (16 * m + (lane & 15)) * kTilePitch + (lane >> 4) * 16);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_bf16(acc[m][n], w[0], w[1], w[2], w[3], x[n / 2][2 * (n & 1)], x[n / 2][2 * (n & 1) + 1]);
                    }
                }
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                __syncthreads();
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sums[warp * (16 * MT * 8 * NT) + (8 * n + 2 * c + (i & 1)) * (16 * MT) + m * 16 + g + 8 * (i >> 1)] = acc[m][n][i];
                __syncthreads();
                for (int i = threadIdx.x; i < 16 * MT * 8 * NT; i += kAdThreads) {
                    const int row = tile0 * 16 + i % (16 * MT), t = i / (16 * MT);
                    if (row >= R || !((tokens >> t) & 1u)) continue;
                    float v = sums[i];
#pragma unroll
                    for (int d = 1; d < kAdWarps; ++d) v += sums[d * (16 * MT * 8 * NT) + i];
                    float* u = a.u + (size_t(split) * a.T + t0 + t) * a.Rp + row;
                    *u = LONG && b0 > s0 ? *u + v : v;  // an element is one thread's every time
                }
                __syncthreads();
            }
        }
    }
}

// Four bf16 of a row of B from j on; zeros from R on (what lies there may be anything).
template <bool VEC> __device__ __forceinline__ uint2 load4(const uint16_t* row, int j, int R) {
    if (j >= R) return make_uint2(0, 0);
    if constexpr (VEC) {
        uint2 v = __ldg(reinterpret_cast<const uint2*>(row + j));
        if (j + 4 > R) {
            if (j + 1 >= R) v.x &= 0xffffu;
            v.y = j + 2 >= R ? 0u : v.y & 0xffffu;
        }
        return v;
    } else {
        const uint32_t w0 = row[j], w1 = j + 1 < R ? row[j + 1] : 0u, w2 = j + 2 < R ? row[j + 2] : 0u,
                       w3 = j + 3 < R ? row[j + 3] : 0u;
        return make_uint2(w0 | (w1 << 16), w2 | (w3 << 16));
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight neighbours of a row of fp32 or bf16 numbers, `n` of them in the row. FAST: 16-byte accesses, n is 8.
template <bool BF16> struct Eight {
    uint32_t w[BF16 ? 4 : 8];
};
template <bool BF16, bool FAST> __device__ __forceinline__ Eight<BF16> load_eight(const void* base, size_t i, int n) {
    Eight<BF16> f;
    if constexpr (FAST) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + i * (BF16 ? 2 : 4));
        const uint4 v = *p;
        f.w[0] = v.x, f.w[1] = v.y, f.w[2] = v.z, f.w[3] = v.w;
        if constexpr (!BF16) {
            const uint4 u = p[1];
            f.w[4] = u.x, f.w[5] = u.y, f.w[6] = u.z, f.w[7] = u.w;
        }
    } else if constexpr (BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + i;
#pragma unroll
        for (int q = 0; q < 4; ++q) f.w[q] = (2 * q < n ? uint32_t(p[2 * q]) : 0u) | (2 * q + 1 < n ? uint32_t(p[2 * q + 1]) << 16 : 0u);
    } else {
        const uint32_t* p = static_cast<const uint32_t*>(base) + i;
#pragma unroll
        for (int q = 0; q < 8; ++q) f.w[q] = q < n ? p[q] : 0u;
    }
    return f;
}
template <bool BF16> __device__ __forceinline__ float of_eight(const Eight<BF16>& f, int q) {
    if constexpr (BF16) return __uint_as_float(q % 2 ? f.w[q / 2] & 0xffff0000u : f.w[q / 2] << 16);
    else return __uint_as_float(f.w[q]);
}
template <bool BF16, bool FAST> __device__ __forceinline__ void store_eight(void* base, size_t i, const float (&v)[8], int n) {
    if constexpr (FAST) {
        char* p = static_cast<char*>(base) + i * (BF16 ? 2 : 4);
        if constexpr (BF16) {
            st_v4(p, make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])));
        } else {
            st_v4(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
            st_v4(p + 16, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < n) {
                if constexpr (BF16) static_cast<uint16_t*>(base)[i + q] = float_to_bf16_bits(v[q]);
                else static_cast<float*>(base)[i + q] = v[q];
            }
    }
}

constexpr int kAdCols = 32;      // columns of a warp's tile: four 8-column operands
constexpr int kAdSteps = 4;      // steps of j whose loads are in flight
constexpr int up_parts(bool out_bf16) { return out_bf16 ? 2 : 3; }
template <int MT> constexpr int up_smem(int Rp, bool out_bf16) { return up_parts(out_bf16) * (Rp / 16) * MT * 32 * 16; }

// Tokens are the 16 rows of an operand here, B's rows its 8 columns: an operand of B is then two neighbouring words of a row, and
// as the columns are dealt a lane has eight neighbouring results of a token, one or two 16-byte accesses of the base and of the
// output. u lies in shared memory in the order of its operand's lanes. (With the rows of B as the 16-row operand its four words
// came from two rows, and five instructions of six were spent on putting them together: 4099 tokens at rank 64 60 us.)
// A warp's tile is 32 columns of one rank's output; per_rank tiles to a rank, and in the column-parallel form the ranks' one
// after the other; `tiles` of them to a CTA. In a step a lane has four j's of a row of B: of S steps together 4 S neighbours.
// FAST: runs of eight columns of base and output are aligned and whole.
template <int MT, int S, bool FAST, bool BASE_BF16, bool OUT_BF16> __global__ void __launch_bounds__(kAdThreads, 2)
k_adapter_up(const __grid_constant__ AdapterArgs a, int slots, int chunks, int tiles, int per_rank) {
    constexpr int kGroup = 16 * MT, kParts = up_parts(OUT_BF16);
    extern __shared__ __align__(128) uint4 s_u[];  // [kParts][steps][MT][32]: what rounding to bf16 leaves, then what it leaves out, ..
    const bool failed = status_failed(a.ctl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t N = uint32_t(a.N);
    const uint32_t b = blockIdx.x / chunks, groups = gridDim.x / chunks / slots;
    const int first = int(blockIdx.x % chunks) * tiles, last = min(first + tiles, a.row ? per_rank : per_rank * a.outs);
    const int sub = slots - 1 - int(b / groups);
    const size_t t0 = size_t(b % groups) * kGroup;
    const int outs = a.row ? a.outs : 1;  // a tile of the row-parallel form goes to every rank
    const Crews crews = crews_of(a, t0, kGroup, true);
    bool waited = false;
    uint32_t todo = crews.firsts;
    for (int crew = 0; todo; ++crew) {
        const int slot = __ffs(todo) - 1;
        todo &= todo - 1;
        if (crew % slots != sub) continue;
        const int adapter = __shfl_sync(0xffffffffu, crews.mine, slot);
        const uint32_t tokens = __shfl_sync(0xffffffffu, crews.same, slot);
        const int R = rank_of(a, adapter), steps = (R + 15) / 16;
        const bool full = S > 1 || (a.b_vec && R % 16 == 0);
        const float scale = R > 0 && a.scale ? a.scale[adapter] : 1.0f;
        const size_t matrix = R > 0 ? size_t(adapter) * a.N * a.R : 0;
        // Fewer tokens than ranks: a token's results go to all lanes, each of which has other ranks: lane (g, c) ranks g, g + 8, ..,
        // token after token. With each lane at its own tokens and the ranks in turn, 32 tokens of 64 adapters over 8 ranks took 18 us.
        const int ntok = __popc(tokens), per = (outs + 7) / 8;
        const bool spread = outs > 1 && ntok <= outs;
        auto turn = [&](int q, int& t, int& k) {  // a lane's q-th token and rank; false if there is none
            const int i = per == 1 ? q : q / per;
            k = g + 8 * (q - i * per);
            if (i >= ntok || k >= outs) return false;
            uint32_t left = tokens;
            for (int d = 0; d < i; ++d) left &= left - 1;
            t = __ffs(left) - 1;
            return true;
        };
        uint2 w[kAdSteps][4];
        Eight<BASE_BF16> base[2 * MT];
        int out0 = 0;    // the tile's first rank and column
        uint32_t n0 = 0;
        auto where = [&](int tile, int& out, uint32_t& n) {
            const int r = a.row ? 0 : tile / per_rank;
            out = a.out0 + r;
            n = uint32_t(tile - r * per_rank) * kAdCols;
        };
        // Operand i's column g is column 8 (g / 2) + 2 i + g % 2 of the tile, so that a lane's results, columns 2c and 2c + 1 of
        // the four operands, are columns 8c to 8c + 7. Rows past the end: the last one.
        auto fetch_rows = [&](int out, uint32_t n, int s0) {
            n += 8 * (g >> 1) + (g & 1);
            const uint16_t* m = a.b[out] + matrix;
            if (FAST) m += size_t(min(n, N - 8 + (g & 1))) * a.R;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint16_t* row = FAST ? m + size_t(2 * i) * a.R : m + size_t(min(n + 2 * i, N - 1)) * a.R;
                if constexpr (S > 1) {
#pragma unroll
                    for (int s = 0; s < kAdSteps; s += 2) {  // two steps' j's in one access: 4 S neighbours of every 16 S
                        const int j = (s0 + s) / S * (16 * S) + 4 * S * c + 4 * (s % S);
                        const uint4 v = j < R ? __ldg(reinterpret_cast<const uint4*>(row + j)) : make_uint4(0, 0, 0, 0);
                        w[s][i] = make_uint2(v.x, v.y);
                        w[s + 1][i] = make_uint2(v.z, v.w);
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < kAdSteps; ++s) {
                        const int j = (s0 + s) * 16 + 4 * c;
                        if (full) w[s][i] = j < R ? __ldg(reinterpret_cast<const uint2*>(row + j)) : make_uint2(0, 0);
                        else if (a.b_vec) w[s][i] = load4<true>(row, j, R);
                        else w[s][i] = load4<false>(row, j, R);
                    }
                }
            }
        };
        // the base of a lane's columns for token t of the group and rank k
        auto fetch_base = [&](int k, uint32_t n, int t, Eight<BASE_BF16>& to) {
            n += 8 * c;
            if (a.has_base && n < N && (tokens >> t) & 1u)
                to = load_eight<BASE_BF16, FAST>(a.base[k], t0 * N + (uint32_t(t) * N + n), int(min(8u, N - n)));
        };
        auto fetch_bases = [&](int k, uint32_t n) {
#pragma unroll
            for (int f = 0; f < 2 * MT; ++f) fetch_base(k, n, 8 * f + g, base[f]);
        };
        auto put = [&](int k, int t, float (&y)[8], const Eight<BASE_BF16>& f) {
            const uint32_t n = n0 + 8 * c;
            if (n >= N || !((tokens >> t) & 1u)) return;
            if (a.has_base)
#pragma unroll
                for (int q = 0; q < 8; ++q) y[q] += of_eight<BASE_BF16>(f, q);
            store_eight<OUT_BF16, FAST>(a.out[k], t0 * N + (uint32_t(t) * N + n), y, int(min(8u, N - n)));
        };
        auto fetch_turn = [&](int q, int out, uint32_t n, Eight<BASE_BF16>& to) {
            int t, k;
            if (turn(q, t, k)) fetch_base(out + k, n, t, to);
        };
        if (first + warp < last) {  // on its way while u is put together
            where(first + warp, out0, n0);
            fetch_rows(out0, n0, 0);
            if (!spread) fetch_bases(out0, n0);
            else
#pragma unroll
                for (int f = 0; f < 2 * MT; ++f) fetch_turn(f, out0, n0, base[f]);
        }
        if (!waited) {
            asm volatile("griddepcontrol.wait;" ::: "memory");  // u is complete
            if (__syncthreads_or(failed)) return;
            waited = true;
        }
        // u: a token to a warp, four j's to a lane
        for (int t = warp; t < kGroup; t += kAdWarps) {
            const bool some = (tokens >> t) & 1u;
            for (int j = 4 * lane; j < 16 * steps; j += 128) {
                float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (some) {
                    const float* u = a.u + (t0 + t) * a.Rp + j;
#pragma unroll 4
                    for (int s = 0; s < a.splits; ++s, u += a.T * a.Rp) {
                        const float4 p = __ldcg(reinterpret_cast<const float4*>(u));
                        v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
                    }
                }
                float y[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) y[q] = j + q < R ? v[q] * scale : 0.0f;  // behind R nothing was written
                // step and lane that have these j's; words 0 and 2 are the first eight tokens', 1 and 3 the second's
                const int in = j % (16 * S), step = j / (16 * S) * S + in % (4 * S) / 4;
                uint32_t* to = reinterpret_cast<uint32_t*>(s_u + (step * MT + t / 16) * 32 + 4 * (t % 8) + in / (4 * S)) + t % 16 / 8;
#pragma unroll
                for (int h = 0; h < kParts; ++h, to += steps * MT * 32 * 4) {
                    to[0] = bf16_pair(y[0], y[1]);
                    to[2] = bf16_pair(y[2], y[3]);
#pragma unroll
                    for (int q = 0; q < 4; ++q)  // an infinity or NaN is in the first part
                        y[q] = fabsf(y[q]) < 3e38f ? y[q] - bf16_bits_to_float(float_to_bf16_bits(y[q])) : 0.0f;
                }
            }
        }
        __syncthreads();
        for (int tile = first + warp; tile < last; tile += kAdWarps) {
            const bool more = tile + kAdWarps < last;
            int next_out = out0;
            uint32_t next_n = n0;
            if (more) where(tile + kAdWarps, next_out, next_n);
            float acc[4][MT][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[i][m][0] = acc[i][m][1] = acc[i][m][2] = acc[i][m][3] = 0.0f;
            for (int s0 = 0; s0 < steps; s0 += kAdSteps) {
                if (s0 > 0) fetch_rows(out0, n0, s0);
                // small parts first: an addition of the matrix instruction cuts what is beyond the sum's last bits
#pragma unroll
                for (int h = kParts - 1; h >= 0; --h)
#pragma unroll
                    for (int s = 0; s < kAdSteps; ++s) {
                        if (s0 + s >= steps) break;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint4 u = s_u[((h * steps + s0 + s) * MT + m) * 32 + lane];
#pragma unroll
                            for (int i = 0; i < 4; ++i) mma_bf16(acc[i][m], u.x, u.y, u.z, u.w, w[s][i].x, w[s][i].y);
                        }
                    }
            }
            if (more) fetch_rows(next_out, next_n, 0);
            if (!spread) {
                for (int k = out0; k < out0 + outs; ++k) {
#pragma unroll
                    for (int f = 0; f < 2 * MT; ++f) {
                        float y[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) y[q] = acc[q / 2][f / 2][2 * (f % 2) + q % 2];
                        put(k, 8 * f + g, y, base[f]);
                        // its place is taken by the next rank's base, or the next tile's
                        if (k + 1 < out0 + outs) fetch_base(k + 1, n0, 8 * f + g, base[f]);
                        else if (more) fetch_base(next_out, next_n, 8 * f + g, base[f]);
                    }
                }
            } else {
                for (int q0 = 0; q0 < ntok * per; q0 += 2 * MT)
#pragma unroll
                    for (int f = 0; f < 2 * MT; ++f) {
                        if (q0 + f >= ntok * per) break;
                        int t = 0, k = 0;
                        const bool some = turn(q0 + f, t, k);
                        const int from = __shfl_sync(0xffffffffu, t, 0);  // lane 0 has a rank in every turn
                        float y[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            y[q] = 0.0f;
#pragma unroll
                            for (int e = 0; e < 2 * MT; ++e) {  // chosen behind the shuffle: a choice among the sums puts them into local memory
                                const float v = __shfl_sync(0xffffffffu, acc[q / 2][e / 2][2 * (e % 2) + q % 2], 4 * (from % 8) + c);
                                if (from / 8 == e) y[q] = v;
                            }
                        }
                        if (some) put(out0 + k, t, y, base[f]);
                        if (q0 + f + 2 * MT < ntok * per) fetch_turn(q0 + f + 2 * MT, out0, n0, base[f]);
                    }
                if (more)
#pragma unroll
                    for (int f = 0; f < 2 * MT; ++f) fetch_turn(f, next_out, next_n, base[f]);
            }
            out0 = next_out;
            n0 = next_n;
        }
        __syncthreads();
    }
}

static size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Tokens of a group: eight while there are few, since then each has an adapter of its own; else 32, since one pass over a matrix
// then serves more of a prompt's tokens. Measured on B200, 4096 x 4096, column-parallel on one rank, us in groups of 8 and of 32: 64 tokens
// of 64 adapters of rank 16 17 and 28, in 8 runs 12 and 16. The border could lie higher: 128 tokens 25 and 39 (in runs 20 and 25), 512 tokens
// 79 and 117 (36 and 53), but 12 adapters in turn 76 and 58.
static int group_tiles(size_t tokens) { return tokens <= 64 ? 1 : 4; }
// CTAs that share a group's adapters: a CTA to each while there are few groups; with many, two, so that a group on the border of two
// requests takes no longer than the others. Measured as above, rank 64, us with a CTA to each and with two: 512 tokens of 12 adapters in
// turn 76 and 132, in 8 runs 68 and 20; 1024 tokens 132 and 174, 69 and 23. What decides is whether a request's tokens follow each other, which
// the host does not know: up to 512 tokens are taken for a batch of single tokens, more for prompts.
static int group_slots(size_t tokens) { return tokens <= 512 ? 8 * group_tiles(tokens) : 2; }

// Parts of the sum over k: as many as give the first kernel a CTA to an SM (two of the form with stages), each of at least 8
// steps or 2 stages; the second kernel waits for all parts (32 tokens of 64 adapters, k 4096, us with 4, 5, 10 and 16 parts: 16.8,
// 17.7, 20.7, 22.3). At least one for 4096 k's, as far as they go: an addition of the matrix instruction cuts what is beyond the sum's
// last bits, always to the same side, and a warp's chain of 64 of them (8192 k's) was off by 1e-6, one of 32 by half of that. Beyond 16 times
// 4096 k's a part's chains end every 4096 (2^22 k's without that were off by 1.5e-4; with more parts instead, as exact, 300 tokens of 8
// adapters of rank 16, 2^20 k's, took 613 us, with chains that end 343, without 255).
// The parts depend on the call's sizes alone, so that a token's sums do not depend on the others' adapters.
int adapter_splits(const AdapterArgs& a, int num_sms) {
    const size_t per = 8 * group_tiles(a.T), groups = (a.T + per - 1) / per, units = a.T <= 512 ? a.T : groups;
    const bool staged = a.x_vec && group_tiles(a.T) > 1;
    const size_t work = staged ? (a.K + kTileK - 1) / kTileK * a.segments / 2 : (a.K + kAdChunk - 1) / kAdChunk * a.segments / 8;
    const size_t least = (a.K * a.segments + kAdChain - 1) / kAdChain;
    return int(std::max<size_t>(1, std::min({std::max(size_t(num_sms) * (staged ? 2 : 1) / units, least), work, size_t(kAdParts)})));
}

template <int NT, int MT, bool LONG> static cudaError_t go_down(const AdapterArgs& a, unsigned ctas, int slots, cudaStream_t s) {
    if constexpr (NT == 4) {
        if (a.x_vec) {
            constexpr int kSmem = kTileStages * tile_bytes<MT>();
            cudaError_t e = cudaFuncSetAttribute(k_adapter_down_tiles<MT, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            if (e != cudaSuccess) return e;
            k_adapter_down_tiles<MT, LONG><<<ctas, kAdThreads, kSmem, s>>>(a, slots);
            return cudaGetLastError();
        }
        k_adapter_down<NT, MT, false, LONG><<<ctas, kAdThreads, 0, s>>>(a, slots);
    } else {
        if (a.x_vec) k_adapter_down<NT, MT, true, LONG><<<ctas, kAdThreads, 0, s>>>(a, slots);
        else k_adapter_down<NT, MT, false, LONG><<<ctas, kAdThreads, 0, s>>>(a, slots);
    }
    return cudaGetLastError();
}

template <int MT> static cudaError_t go_up(const AdapterArgs& a, int num_sms, cudaStream_t s) {
    const size_t groups = (a.T + 16 * MT - 1) / (16 * MT), slots = a.T <= 512 ? 16 * MT : 2;
    // tiles of a CTA: as many to each warp as leave two CTAs to an SM
    const size_t units = a.T <= 512 ? a.T : groups, per_rank = (a.N + kAdCols - 1) / kAdCols, all = per_rank * (a.row ? 1 : a.outs);
    if (all > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    const size_t share = std::max<size_t>(1, size_t(2 * num_sms) / units), tiles = round_up((all + share - 1) / share, kAdWarps);
    const size_t chunks = (all + tiles - 1) / tiles, ctas = groups * slots * chunks;
    if (ctas > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    bool fast = a.N % 8 == 0;
    for (int r = a.out0; r < a.out0 + a.outs; ++r)
        fast = fast && reinterpret_cast<uintptr_t>(a.out[r]) % 16 == 0 && reinterpret_cast<uintptr_t>(a.base[r]) % 16 == 0;
    // rows of B in 16-byte accesses where every adapter has all of max_rank, 32 or 64 j's at a time
    bool b16 = !a.rank && a.R % 32 == 0;
    for (int r = a.out0; r < a.out0 + (a.row ? 1 : a.outs); ++r) b16 = b16 && reinterpret_cast<uintptr_t>(a.b[r]) % 16 == 0;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(ctas));
    cfg.blockDim = dim3(kAdThreads);
    cfg.dynamicSmemBytes = size_t(up_smem<MT>(a.Rp, a.out_bf16));  // 48 KiB at most
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    auto go = [&](auto kernel) {
        if (cfg.dynamicSmemBytes > 47 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(cfg.dynamicSmemBytes));
            if (e != cudaSuccess) return e;
        }
        return cudaLaunchKernelEx(&cfg, kernel, a, int(slots), int(chunks), int(tiles), int(per_rank));
    };
    auto types = [&](auto at_once, auto aligned) {
        constexpr int S = decltype(at_once)::value;
        constexpr bool F = decltype(aligned)::value;
        if (a.base_bf16) return a.out_bf16 ? go(k_adapter_up<MT, S, F, true, true>) : go(k_adapter_up<MT, S, F, true, false>);
        return a.out_bf16 ? go(k_adapter_up<MT, S, F, false, true>) : go(k_adapter_up<MT, S, F, false, false>);
    };
    if (!fast) return types(std::integral_constant<int, 1>{}, std::false_type{});
    if (b16) return a.R % 64 == 0 ? types(std::integral_constant<int, 4>{}, std::true_type{}) : types(std::integral_constant<int, 2>{}, std::true_type{});
    return types(std::integral_constant<int, 1>{}, std::true_type{});
}

template <int NT> static cudaError_t go_adapters(const AdapterArgs& a, int num_sms, cudaStream_t s) {
    const int slots = group_slots(a.T);
    const size_t groups = (a.T + 8 * NT - 1) / (8 * NT), down = groups * slots * a.splits;
    if (down > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    auto ranks = [&](auto chains) {
        constexpr bool LONG = decltype(chains)::value;
        return a.R <= 16 ? go_down<NT, 1, LONG>(a, unsigned(down), slots, s) : a.R <= 32 ? go_down<NT, 2, LONG>(a, unsigned(down), slots, s)
                                                                                       : go_down<NT, 4, LONG>(a, unsigned(down), slots, s);
    };
    // in the same kernels the ends of chains cost 4,099 tokens at rank 64, k 4096, 1 us of 48
    cudaError_t e = a.K * a.segments > size_t(kAdParts) * kAdChain ? ranks(std::true_type{}) : ranks(std::false_type{});
    return e != cudaSuccess ? e : go_up<NT == 1 ? 1 : 2>(a, num_sms, s);
}

cudaError_t launch_adapters(const AdapterArgs& a, int num_sms, cudaStream_t s) {
    return group_tiles(a.T) == 1 ? go_adapters<1>(a, num_sms, s) : go_adapters<4>(a, num_sms, s);
}

}  // namespace simcomm
