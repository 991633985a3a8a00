// Few tokens times a matrix of 4-bit weights with group scales, its shards on the communicator's ranks.
//
//   W[n][k] = (q[n][k] - 8) * scale[n][k / group]
//   column parallel  rank r holds rows [r N/p, (r+1) N/p) of W and a copy of x: out[r] = x[r] W_r^T
//   row parallel     rank r holds columns [r K/p, (r+1) K/p) of W and of x: out[q] = sum_r x[r] W_r^T
//                    on every rank q (the AllReduce of the ranks' partial products)
//
// In the row-parallel form the exchange costs nothing of its own: the sum over ranks is part of the sum
// over k, whose range one CTA's warps split between them, and the epilogue stores the finished value to
// every rank's output. Bound by the weights' bytes; the warp-level product is in wprod.cuh.
#include <algorithm>

#include "wprod.cuh"

namespace simcomm {

constexpr int kLinWarps = 8;
constexpr int kLinThreads = kLinWarps * 32;

template <bool BF16> __device__ __forceinline__ void st_out(void* p, size_t i, float v) {
    if constexpr (BF16) static_cast<uint16_t*>(p)[i] = float_to_bf16_bits(v);
    else static_cast<float*>(p)[i] = v;
}

template <int WK, bool VEC, int NT>
__global__ void __launch_bounds__(kLinThreads, 2) k_linear_q4(const __grid_constant__ LinearArgs a) {
    using W = WTraits<WK>;
    __shared__ float s_red[kLinWarps][4 * NT][32];
    if (status_failed(a.ctl)) return;  // one word, the same for the whole CTA unless it is being set
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // CTA -> (rank of a column-parallel call, block of row tiles, token tile); token tiles of one block
    // are neighbours, so the second reads the block's weights from L2
    uint32_t u = blockIdx.x;
    const int tt = int(u % a.token_tiles);
    u /= a.token_tiles;
    const size_t blk = u % a.tile_blocks;
    const int rank0 = a.row ? 0 : (a.view_rank >= 0 ? a.view_rank : int(u / a.tile_blocks));
    const int per = kLinWarps / a.splits, split = warp % a.splits;
    const size_t row0 = (blk * per + warp / a.splits) * 16;
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    if (row0 < a.N) {
        const int cpr = int(a.K / W::kChunk);  // chunks of one rank's row
        const int total = cpr * (a.row ? a.p : 1);
        const int lo = int((long long)total * split / a.splits), hi = int((long long)total * (split + 1) / a.splits);
        const size_t wrow = a.K / 2, srow = a.K >> a.group_shift;
        const size_t r0 = row0 + g, r1 = row0 + g + 8;
        for (int c = lo; c < hi;) {
            const int q = c / cpr, rank = rank0 + q;
            const int end = min(hi, (q + 1) * cpr);
            LaneRows rows;
            rows.w0 = r0 < a.N ? a.w[rank] + r0 * wrow : nullptr;
            rows.w1 = r1 < a.N ? a.w[rank] + r1 * wrow : nullptr;
            rows.s0 = a.scale[rank] + r0 * srow;
            rows.s1 = a.scale[rank] + r1 * srow;
            const uint16_t* x[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const size_t tok = size_t(tt) * (8 * NT) + n * 8 + g;
                x[n] = tok < a.T ? a.x[rank] + tok * a.K : nullptr;
            }
            warp_product<WK, VEC, NT>(acc, rows, x, c - q * cpr, end - q * cpr, int(a.K), a.chunk_shift, t);
            c = end;
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_red[warp][4 * n + i][lane] = acc[n][i];
    __syncthreads();
    // every element of the CTA's tiles: the sum over its warps in order, stored to the ranks that get it
    const int first = a.row ? (a.view_rank >= 0 ? a.view_rank : 0) : rank0;
    const int last = a.row ? (a.view_rank >= 0 ? a.view_rank + 1 : a.p) : rank0 + 1;
    for (int e = threadIdx.x; e < per * 16 * 8 * NT; e += kLinThreads) {
        const int r = e % 16, tok = (e / 16) % (8 * NT), q = e / (16 * 8 * NT);
        const size_t row = (blk * per + q) * 16 + r;
        const size_t token = size_t(tt) * (8 * NT) + tok;
        if (row >= a.N || token >= a.T) continue;
        const int reg = 4 * (tok / 8) + (r / 8) * 2 + (tok & 1), ln = (r % 8) * 4 + (tok % 8) / 2;
        float v = s_red[q * a.splits][reg][ln];
        for (int s = 1; s < a.splits; ++s) v += s_red[q * a.splits + s][reg][ln];
        for (int d = first; d < last; ++d) {
            if (a.out_bf16) st_out<true>(a.out[d], token * a.N + row, v);
            else st_out<false>(a.out[d], token * a.N + row, v);
        }
    }
}

template <int WK>
static cudaError_t launch_linear_kind(LinearArgs& a, int nt, unsigned grid, cudaStream_t s) {
    auto go = [&](auto kernel) {
        kernel<<<grid, kLinThreads, 0, s>>>(a);
        return cudaGetLastError();
    };
    if (a.x_vec) return nt == 1 ? go(k_linear_q4<WK, true, 1>) : nt == 2 ? go(k_linear_q4<WK, true, 2>) : go(k_linear_q4<WK, true, 4>);
    return nt == 1 ? go(k_linear_q4<WK, false, 1>) : nt == 2 ? go(k_linear_q4<WK, false, 2>) : go(k_linear_q4<WK, false, 4>);
}

cudaError_t launch_linear(const LinearArgs& args, int num_sms, cudaStream_t s) {
    LinearArgs a = args;
    const int nt = a.T <= 8 ? 1 : a.T <= 16 ? 2 : 4;
    const size_t tiles = (a.N + 15) / 16;
    a.token_tiles = uint32_t((a.T + 8 * nt - 1) / (8 * nt));
    const size_t jobs = tiles * a.token_tiles * (a.row || a.view_rank >= 0 ? 1 : size_t(a.p));
    // warps of a CTA on one row tile: more, the fewer tiles there are to fill the GPU with
    int splits = 1;
    while (splits < kLinWarps && jobs * splits < size_t(num_sms) * 8 * kLinWarps) splits *= 2;
    a.splits = splits;
    const size_t per = kLinWarps / splits;
    a.tile_blocks = uint32_t((tiles + per - 1) / per);
    const size_t ctas = size_t(a.tile_blocks) * a.token_tiles * (a.row || a.view_rank >= 0 ? 1 : size_t(a.p));
    if (ctas > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    const int group = 1 << a.group_shift;
    a.chunk_shift = 0;
    while ((128 << a.chunk_shift) < group) ++a.chunk_shift;
    if (group >= 128) return launch_linear_kind<W_Q4X4>(a, nt, unsigned(ctas), s);
    if (group == 64) return launch_linear_kind<W_Q4X2>(a, nt, unsigned(ctas), s);
    return launch_linear_kind<W_Q4X1>(a, nt, unsigned(ctas), s);
}

}  // namespace simcomm
