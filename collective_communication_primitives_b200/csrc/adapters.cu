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
// without shared memory.
//
// u is fp32, its parts over k joined in order by the second kernel, which splits it into two bf16 parts (what is lost is
// 2^-16 of it or less) since B u would otherwise carry a rounding of 2^-9. Bound by the bytes of the tokens, outputs and
// met adapters; in a decode step by the latency of two kernels that wait for two loads each.
#include <algorithm>

#include "common.cuh"
#include "wprod.cuh"

namespace simcomm {

constexpr int kAdThreads = 256;
constexpr int kAdWarps = kAdThreads / 32;
constexpr int kAdChunk = 32;   // k's of one step of k_adapter_down: two matrix instructions
constexpr int kAdAhead = 4;    // steps whose loads are in flight

// A group's tokens that have the adapter of its token `slot`, if that is the first such token.
struct Crew {
    int adapter;      // -1: none
    uint32_t tokens;  // a bit each; 0: nothing to do
};
__device__ __forceinline__ Crew crew_of(const AdapterArgs& a, size_t t0, int group, int slot, bool none_too) {
    const int lane = threadIdx.x & 31;
    const bool here = lane < group && t0 + lane < a.T;
    int e = here ? a.adapter[t0 + lane] : -2;
    if (here && (e < -1 || e >= a.adapters)) {
        raise_status(a.ctl, COLL_ERR_INVALID_ARG);
        e = -1;
    }
    const int mine = __shfl_sync(0xffffffffu, e, slot);
    const uint32_t same = __ballot_sync(0xffffffffu, e == mine);
    const bool first = (same & ((1u << slot) - 1u)) == 0u;
    return Crew{mine, first && (mine >= 0 || (mine == -1 && none_too)) ? same : 0u};
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

// NT: tokens of a group in eights. The CTA's warps share the rows of A, 16 to a tile, and, where there are fewer tiles than
// warps, the steps of k.
template <int NT, bool VEC> __global__ void __launch_bounds__(kAdThreads, 2)
k_adapter_down(const __grid_constant__ AdapterArgs a, int slots) {
    __shared__ float s_sum[kAdWarps][16 * 8 * NT];
    if (__syncthreads_or(status_failed(a.ctl))) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    size_t b = blockIdx.x;
    const int split = int(b % a.splits);
    b /= a.splits;
    const int sub = int(b % slots);
    const size_t t0 = b / slots * (8 * NT);
    const uint32_t steps = uint32_t((a.K + kAdChunk - 1) / kAdChunk), all = steps * a.segments;
    const uint32_t s0 = uint32_t(uint64_t(all) * split / a.splits), s1 = uint32_t(uint64_t(all) * (split + 1) / a.splits);
    for (int slot = sub; slot < 8 * NT; slot += slots) {
        const Crew crew = crew_of(a, t0, 8 * NT, slot, false);
        if (!crew.tokens) continue;
        const int R = rank_of(a, crew.adapter), tiles = (R + 15) / 16;
        int wide = 1;  // warps side by side on tiles of rows
        while (wide < tiles && wide < kAdWarps) wide *= 2;
        const int deep = kAdWarps / wide, turn = warp / wide;  // warps on each tile, one behind the other in k
        for (int tile0 = 0; tile0 < tiles; tile0 += wide) {
            const int tile = tile0 + warp % wide;
            float acc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
            if (tile < tiles) {
                const size_t e = size_t(crew.adapter) * a.R;
                const size_t r0 = (e + min(tile * 16 + g, R - 1)) * a.K, r1 = (e + min(tile * 16 + g + 8, R - 1)) * a.K;
                for (uint32_t s = s0 + turn; s < s1; s += deep * kAdAhead) {
                    uint4 w[kAdAhead][2], x[kAdAhead][NT];
#pragma unroll
                    for (int q = 0; q < kAdAhead; ++q) {
                        const uint32_t at = s + q * deep;
                        const uint32_t seg = at < s1 ? at / steps : 0u;
                        const size_t k = at < s1 ? size_t(at - seg * steps) * kAdChunk + c * 8 : a.K;
                        const uint16_t* m = a.a[a.rank0 + seg];
                        const uint16_t* v = a.x[a.rank0 + seg];
                        w[q][0] = load8<VEC>(m + r0, k, a.K);
                        w[q][1] = load8<VEC>(m + r1, k, a.K);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            x[q][n] = (crew.tokens >> (8 * n + g)) & 1u ? load8<VEC>(v + (t0 + 8 * n + g) * a.K, k, a.K)
                                                                         : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int q = 0; q < kAdAhead; ++q)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_bf16(acc[n], w[q][0].x, w[q][1].x, w[q][0].y, w[q][1].y, x[q][n].x, x[q][n].y);
                            mma_bf16(acc[n], w[q][0].z, w[q][1].z, w[q][0].w, w[q][1].w, x[q][n].z, x[q][n].w);
                        }
                }
            }
            // row g or g + 8 of the tile, tokens 2c and 2c + 1 of eight n
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s_sum[warp][(8 * n + 2 * c + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[n][i];
            __syncthreads();
            for (int i = threadIdx.x; i < wide * 16 * 8 * NT; i += kAdThreads) {
                const int j = i % (16 * wide), t = i / (16 * wide), row = tile0 * 16 + j;
                if (row < R && (crew.tokens >> t) & 1u) {
                    float v = 0.0f;
                    for (int d = 0; d < deep; ++d) v += s_sum[d * wide + j / 16][t * 16 + j % 16];
                    a.u[(size_t(split) * a.T + t0 + t) * a.Rp + row] = v;
                }
            }
            __syncthreads();
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

template <bool BF16> __device__ __forceinline__ float2 load_pair(const void* base, size_t i, bool two, bool aligned) {
    if constexpr (BF16) {
        if (aligned) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + i);
            return make_float2(bf16_bits_to_float(w & 0xffffu), bf16_bits_to_float(w >> 16));
        }
        const uint16_t* p = static_cast<const uint16_t*>(base) + i;
        return make_float2(bf16_bits_to_float(p[0]), two ? bf16_bits_to_float(p[1]) : 0.0f);
    } else {
        const float* p = static_cast<const float*>(base) + i;
        if (aligned) return *reinterpret_cast<const float2*>(p);
        return make_float2(p[0], two ? p[1] : 0.0f);
    }
}
template <bool BF16> __device__ __forceinline__ void store_pair(void* base, size_t i, float2 v, bool two, bool aligned) {
    if constexpr (BF16) {
        uint16_t* p = static_cast<uint16_t*>(base) + i;
        const uint32_t lo = float_to_bf16_bits(v.x), hi = float_to_bf16_bits(v.y);
        if (aligned) {
            *reinterpret_cast<uint32_t*>(p) = lo | (hi << 16);
        } else {
            p[0] = uint16_t(lo);
            if (two) p[1] = uint16_t(hi);
        }
    } else {
        float* p = static_cast<float*>(base) + i;
        if (aligned) {
            *reinterpret_cast<float2*>(p) = v;
        } else {
            p[0] = v.x;
            if (two) p[1] = v.y;
        }
    }
}

constexpr int kAdStride = kAdapterMaxRank + 16;  // of a token's u in shared memory: half a warp's 8-byte reads meet 32 banks

// pairs: two columns of out and base that follow each other are one aligned access. n_cta: columns of a CTA.
template <int NT, bool VEC, bool BASE_BF16, bool OUT_BF16> __global__ void __launch_bounds__(kAdThreads, 2)
k_adapter_up(const __grid_constant__ AdapterArgs a, int slots, int chunks, int n_cta, int pairs) {
    __shared__ __align__(8) uint16_t s_u[2][8 * NT][kAdStride];  // what rounding to bf16 leaves, and what it leaves out
    if (__syncthreads_or(status_failed(a.ctl))) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    size_t b = blockIdx.x;
    const size_t first = b % chunks * n_cta;
    b /= chunks;
    const int shard = a.row ? 0 : int(b % a.outs);  // a column-parallel CTA is one rank's
    if (!a.row) b /= a.outs;
    const int sub = int(b % slots);
    const size_t t0 = b / slots * (8 * NT);
    const int out0 = a.out0 + shard, outs = a.row ? a.outs : 1;
    for (int slot = sub; slot < 8 * NT; slot += slots) {
        const Crew crew = crew_of(a, t0, 8 * NT, slot, true);
        if (!crew.tokens) continue;
        const int R = rank_of(a, crew.adapter), steps = (R + 15) / 16;
        const float scale = R > 0 && a.scale ? a.scale[crew.adapter] : 1.0f;
        for (int i = threadIdx.x; i < steps * 16 * 8 * NT; i += kAdThreads) {
            const int j = i % (16 * steps), t = i / (16 * steps);
            float v = 0.0f;
            if (j < R && (crew.tokens >> t) & 1u) {
                for (int s = 0; s < a.splits; ++s) v += __ldcg(a.u + (size_t(s) * a.T + t0 + t) * a.Rp + j);
                v *= scale;
            }
            const uint16_t hi = float_to_bf16_bits(v);
            const float left = v - bf16_bits_to_float(hi);
            s_u[0][t][j] = hi;
            s_u[1][t][j] = fabsf(v) < 3e38f ? float_to_bf16_bits(left) : uint16_t(0);  // an infinity or NaN is in the first part
        }
        __syncthreads();
        const uint16_t* m = a.b[out0] + (R > 0 ? size_t(crew.adapter) * a.N * a.R : 0);
        for (size_t n0 = first + warp * 16; n0 < min(a.N, first + n_cta); n0 += kAdWarps * 16) {
            // a lane's results are columns n and n + 1 of tokens 2c and 2c + 1 of every eight: rows 2g and 2g + 1 of B lie in the
            // instruction's rows g and g + 8
            const size_t n = n0 + 2 * g;
            const bool in = n < a.N, two = n + 1 < a.N;
            const uint16_t* r0 = m + min(n, a.N - 1) * a.R;
            const uint16_t* r1 = m + min(n + 1, a.N - 1) * a.R;
            float acc[NT][4];
#pragma unroll
            for (int q = 0; q < NT; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.0f;
            for (int s = 0; s < steps; ++s) {
                const uint2 w0 = load4<VEC>(r0, s * 16 + 4 * c, R), w1 = load4<VEC>(r1, s * 16 + 4 * c, R);
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint2 u = *reinterpret_cast<const uint2*>(&s_u[h][8 * q + g][s * 16 + 4 * c]);
                        mma_bf16(acc[q], w0.x, w1.x, w0.y, w1.y, u.x, u.y);
                    }
            }
            if (in)
                for (int k = out0; k < out0 + outs; ++k) {
                    float2 base[NT][2];
#pragma unroll
                    for (int q = 0; q < NT; ++q)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int t = 8 * q + 2 * c + i;
                            base[q][i] = a.has_base && (crew.tokens >> t) & 1u
                                             ? load_pair<BASE_BF16>(a.base[k], (t0 + t) * a.N + n, two, pairs)
                                             : make_float2(0.0f, 0.0f);
                        }
#pragma unroll
                    for (int q = 0; q < NT; ++q)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int t = 8 * q + 2 * c + i;
                            if (!((crew.tokens >> t) & 1u)) continue;
                            store_pair<OUT_BF16>(a.out[k], (t0 + t) * a.N + n,
                                                 make_float2(base[q][i].x + acc[q][i], base[q][i].y + acc[q][2 + i]), two, pairs);
                        }
                }
        }
        __syncthreads();
    }
}

// Tokens of a group: eight while there are few, since then each has an adapter of its own; else 32, since one pass over a matrix
// then serves more of a prompt's tokens.
static int group_tiles(size_t tokens) { return tokens <= 64 ? 1 : 4; }
// CTAs that share a group's adapters: all apart while there are few groups, together when there are many.
static int group_slots(size_t tokens) { return tokens <= 512 ? 8 * group_tiles(tokens) : 1; }

// Parts of the sum over k: as many as give two CTAs to an SM, each of at least 8 steps. They depend on the call's sizes
// alone, so that a token's sums do not depend on the others' adapters.
int adapter_splits(size_t tokens, size_t k, int segments, int num_sms) {
    const size_t groups = (tokens + 8 * group_tiles(tokens) - 1) / (8 * group_tiles(tokens));
    const size_t units = tokens <= 512 ? tokens : groups, steps = (k + kAdChunk - 1) / kAdChunk * segments;
    return int(std::max<size_t>(1, std::min({(size_t(2 * num_sms) + units - 1) / units, steps / 8, size_t(16)})));
}

template <int NT> static cudaError_t go_adapters(const AdapterArgs& a, int num_sms, cudaStream_t s) {
    const int slots = group_slots(a.T);
    const size_t groups = (a.T + 8 * NT - 1) / (8 * NT), down = groups * slots * a.splits;
    // columns of a CTA of the second kernel: in 128s, as many as leave four CTAs to an SM
    const size_t units = (a.T <= 512 ? a.T : groups) * (a.row ? 1 : a.outs);
    size_t n_cta = 128;
    while (n_cta < 1024 && units * ((a.N + 2 * n_cta - 1) / (2 * n_cta)) >= size_t(4 * num_sms)) n_cta *= 2;
    const size_t chunks = (a.N + n_cta - 1) / n_cta, up = groups * slots * chunks * (a.row ? 1 : a.outs);
    if (down > size_t(INT32_MAX) || up > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    if (a.x_vec) k_adapter_down<NT, true><<<unsigned(down), kAdThreads, 0, s>>>(a, slots);
    else k_adapter_down<NT, false><<<unsigned(down), kAdThreads, 0, s>>>(a, slots);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    bool pairs = a.N % 2 == 0;
    const size_t bo = a.out_bf16 ? 4 : 8, bb = a.base_bf16 ? 4 : 8;
    for (int r = a.out0; r < a.out0 + a.outs; ++r)
        pairs = pairs && reinterpret_cast<uintptr_t>(a.out[r]) % bo == 0 && reinterpret_cast<uintptr_t>(a.base[r]) % bb == 0;
    auto go = [&](auto kernel) {
        kernel<<<unsigned(up), kAdThreads, 0, s>>>(a, slots, int(chunks), int(n_cta), pairs ? 1 : 0);
        return cudaGetLastError();
    };
    auto types = [&](auto vec) {
        constexpr bool V = decltype(vec)::value;
        if (a.base_bf16) return a.out_bf16 ? go(k_adapter_up<NT, V, true, true>) : go(k_adapter_up<NT, V, true, false>);
        return a.out_bf16 ? go(k_adapter_up<NT, V, false, true>) : go(k_adapter_up<NT, V, false, false>);
    };
    return a.b_vec ? types(std::true_type{}) : types(std::false_type{});
}

cudaError_t launch_adapters(const AdapterArgs& a, int num_sms, cudaStream_t s) {
    return group_tiles(a.T) == 1 ? go_adapters<1>(a, num_sms, s) : go_adapters<4>(a, num_sms, s);
}

}  // namespace simcomm
