// Few tokens times a matrix of 4-bit weights with group scales, its shards on the communicator's ranks.
//
//   W[n][k] = (q[n][k] - 8) * scale[n][k / group]
//   column parallel  rank r holds rows [r N/p, (r+1) N/p) of W and a copy of x: out[r] = x[r] W_r^T
//   row parallel     rank r holds columns [r K/p, (r+1) K/p) of W and of x: out[q] = sum_r x[r] W_r^T
//                    on every rank q (the AllReduce of the ranks' partial products)
//
// In the row-parallel form the exchange costs nothing of its own: the sum over ranks is part of the sum
// over k, whose range one CTA's warps split between them, and the epilogue stores the finished value to
// every rank's output. The warp-level product and what bounds it are in wprod.cuh. Measured on B200: 4096 x 4096, one
// token, row parallel over 8 ranks 13.5 us (the bytes take 1.4 at the copy rate: every rank's tokens are a panel of their
// own, half empty, and go through two buffers one after the other); 65536 x 4096, one token 47 us (21.6); 131072 x 4096,
// 16 tokens 117 us, 2.5 TB/s (45); 16384 x 4096, 512 tokens 316 us (13.2: the weights are taken apart for every 32).
#include <algorithm>
#include <type_traits>

#include "wprod.cuh"

namespace simcomm {

template <bool BF16> __device__ __forceinline__ void st_out(void* p, size_t i, float v) {
    if constexpr (BF16) static_cast<uint16_t*>(p)[i] = float_to_bf16_bits(v);
    else static_cast<float*>(p)[i] = v;
}

// Unit -> (rank of a column-parallel call, block of row tiles, token tile); token tiles of one block are
// neighbours, so that the second reads the block's weights from L2. Units from tail_first on are pieces of a
// block: of its row tiles, each shared by as many times more warps.
template <int WK, bool VEC, int MT, int NT> struct LinearJob {
    static constexpr int kWK = WK, kMT = MT;
    static constexpr bool kVecW = true, kVecX = VEC;
    static constexpr ptrdiff_t part = 0;
    const LinearArgs& a;
    int K, segments, chunk_shift;

    __device__ __forceinline__ int split_shift(int u) const { return a.shift + (u >= a.tail_first ? a.tail_shift : 0); }
    struct At { int rank; size_t row0, token0; };  // of the unit's first segment
    __device__ __forceinline__ At at(int u) const {
        At x;
        const int shift = split_shift(u);
        int piece = 0;
        if (u >= a.tail_first) {
            piece = (u - a.tail_first) & ((1 << a.tail_shift) - 1);
            u = a.tail_first + ((u - a.tail_first) >> a.tail_shift);
        }
        x.token0 = size_t(uint32_t(u) % a.token_tiles) * (8 * NT);
        const uint32_t b = uint32_t(u) / a.token_tiles;
        x.row0 = size_t(b % a.tile_blocks) * (kProdWarps >> a.shift) * (16 * MT) + piece * (kProdWarps >> shift) * (16 * MT);
        x.rank = a.row ? 0 : a.view_rank >= 0 ? a.view_rank : int(b / a.tile_blocks);
        return x;
    }
    __device__ __forceinline__ size_t row_at(const At& x, int tile, int r) const {  // rows past the end: the last one
        return min(x.row0 + tile * (16 * MT) + r, a.N - 1);
    }
    __device__ __forceinline__ void rows(int u, int seg, int tile, int g, const char* (&w)[MT][2]) const {
        const At x = at(u);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) w[m][i] = a.w[x.rank + seg] + row_at(x, tile, m * 16 + i * 8 + g) * (a.K / 2);
    }
    __device__ __forceinline__ void scales(int u, int seg, int tile, int g, int t, const uint16_t* (&s)[(MT + 1) / 2]) const {
        const At x = at(u);
#pragma unroll
        for (int q = 0; q < (MT + 1) / 2; ++q)
            s[q] = a.scale[x.rank + seg] +
                   row_at(x, tile, (2 * q + (MT > 1 ? t / 2 : 0)) * 16 + t % 2 * 8 + g) * (a.K >> a.group_shift);
    }
    __device__ __forceinline__ const uint16_t* token(int u, int seg, int n) const {
        const At x = at(u);
        return x.token0 + n < a.T ? a.x[x.rank + seg] + (x.token0 + n) * a.K : nullptr;
    }
};

template <int WK, bool VEC, int MT, int NT>
__global__ void __launch_bounds__(kProdThreads, 1) k_linear_q4(const __grid_constant__ LinearArgs a) {
    extern __shared__ __align__(128) unsigned char s_raw[];
    __shared__ int s_fail;
    const ProductSmem s = product_layout<MT, 1>(s_raw);
    if (threadIdx.x == 0) {
        s_fail = status_failed(a.ctl);
        init_panels(s);
    }
    __syncthreads();
    if (s_fail) return;
    using Job = LinearJob<WK, VEC, MT, NT>;
    const Job job{a, int(a.K), a.row ? a.p : 1, a.chunk_shift};
    PanelCount pc;
    if (threadIdx.x >= kProdWarps * 32) {
        for (int u = blockIdx.x; u < a.units; u += gridDim.x)
            if (!copy_tokens<NT, 1>(job, a.ctl, a.timeout_ns, s, pc, u)) break;
        land_panels(a.ctl, s, pc);
        return;
    }
    Multiplier<Job> mul(job, s, blockIdx.x, a.units, gridDim.x);
    if (int(blockIdx.x) == a.fault_cta && threadIdx.x < 32) mul.give_up();
    for (int u = blockIdx.x; u < a.units; u += gridDim.x) {
        float acc[MT][NT][4];
        mul.template unit<NT, 1>(a.ctl, a.timeout_ns, pc, u, acc);
        const typename Job::At x = job.at(u);
        // stored to the ranks that get it
        const int first = a.row ? (a.view_rank >= 0 ? a.view_rank : 0) : x.rank;
        const int last = a.row ? (a.view_rank >= 0 ? a.view_rank + 1 : a.p) : x.rank + 1;
        finish_unit<false, MT, NT>(s, 1 << job.split_shift(u), acc, [&](int tile, int r, int c, float v, float) {
            const size_t row = x.row0 + tile * (16 * MT) + r, token = x.token0 + c;
            if (row >= a.N || token >= a.T || !mul.live) return;
            for (int d = first; d < last; ++d) {
                if (a.out_bf16) st_out<true>(a.out[d], token * a.N + row, v);
                else st_out<false>(a.out[d], token * a.N + row, v);
            }
        });
    }
    mul.drain(a.ctl);
}

template <int WK, int MT, int NT> static cudaError_t launch_linear_kind(const LinearArgs& a, int num_sms, cudaStream_t s) {
    auto go = [&](auto kernel) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, product_smem<MT, 1>());
        if (e != cudaSuccess) return e;
        const unsigned grid = unsigned(std::min(a.units, num_sms));
        kernel<<<grid, kProdThreads, product_smem<MT, 1>(), s>>>(a);
        return cudaGetLastError();
    };
    return a.x_vec ? go(k_linear_q4<WK, true, MT, NT>) : go(k_linear_q4<WK, false, MT, NT>);
}

cudaError_t launch_linear(const LinearArgs& args, int num_sms, cudaStream_t s) {
    LinearArgs a = args;
    const int nt = a.T <= 8 ? 1 : a.T <= 16 ? 2 : 4;
    a.token_tiles = uint32_t((a.T + 8 * nt - 1) / (8 * nt));
    const size_t shards = a.row || a.view_rank >= 0 ? 1 : size_t(a.p);
    // Row tiles of a warp: two use every staged token twice, one spreads few rows over more warps. Measured on B200,
    // one and two: 12.4 and 14.4 us at 4096 x 4096 with 16 tokens, 26.8 and 24.7 at 16384 x 4096, 146 and 129 at
    // 131072 x 4096.
    const size_t units = (a.N + 15) / 16 * a.token_tiles * shards, warps = size_t(num_sms) * kProdWarps;
    const int mt = units * 4 >= warps ? 2 : 1;
    const size_t tiles = (a.N + 16 * mt - 1) / (16 * mt), jobs = tiles * a.token_tiles * shards;
    // Warps of a CTA on one row tile: as many as give half the GPU's warps work. More mean fewer rows per CTA, so that
    // the same tokens are staged more often. Measured on B200 with 1, 2, 4 and 8 of them: 22.6, 16.5, 12.4, 12.4 us at
    // 4096 x 4096 with one token, 24.8, 28.8, 32.8, 34.9 at 32768 x 4096, and 49 and 66 with 1 and 2 at 16384 x 4096
    // with 64 tokens.
    const int group = 1 << a.group_shift;
    const int stages = int(a.K / 128), panel = kPanelK / nt / 128;
    a.shift = 0;
    while ((1 << a.shift) < std::min(kProdWarps, panel) && (2 << a.shift) <= stages &&
           (jobs << a.shift) * 2 < size_t(num_sms) * kProdWarps)
        ++a.shift;
    const size_t per = kProdWarps >> a.shift;
    const size_t blocks = (tiles + per - 1) / per, ctas = blocks * a.token_tiles * shards;
    if (ctas > size_t(INT32_MAX) / 2) return cudaErrorInvalidValue;  // unit numbers step past the last by a grid
    // A last round that less than fills the GPU is cut into pieces, more warps to a row tile: measured on B200 129
    // and 117 us at 131072 x 4096 with 16 tokens (3.46 rounds), 64 and 51 at 50256 x 4096 (1.35), without and with it.
    const int rest = int(ctas % size_t(num_sms));
    a.tail_shift = 0;
    while (ctas > size_t(num_sms) && rest && (rest << a.tail_shift) * 2 <= num_sms &&
           (2 << (a.shift + a.tail_shift)) <= std::min({kProdWarps, panel, stages / 2}))
        ++a.tail_shift;
    a.tail_first = int(ctas) - rest;
    a.units = a.tail_first + (rest << a.tail_shift);
    a.tile_blocks = uint32_t(blocks);
    a.chunk_shift = 0;
    while ((128 << a.chunk_shift) < group) ++a.chunk_shift;
    auto kind = [&](auto wk) {
        constexpr int WK = decltype(wk)::value;
        if (mt == 1)
            return nt == 1 ? launch_linear_kind<WK, 1, 1>(a, num_sms, s) : nt == 2 ? launch_linear_kind<WK, 1, 2>(a, num_sms, s)
                                                                                : launch_linear_kind<WK, 1, 4>(a, num_sms, s);
        return nt == 1 ? launch_linear_kind<WK, 2, 1>(a, num_sms, s) : nt == 2 ? launch_linear_kind<WK, 2, 2>(a, num_sms, s)
                                                                            : launch_linear_kind<WK, 2, 4>(a, num_sms, s);
    };
    if (group >= 128) return kind(std::integral_constant<int, W_Q4X4>());
    if (group == 64) return kind(std::integral_constant<int, W_Q4X2>());
    return kind(std::integral_constant<int, W_Q4X1>());
}

}  // namespace simcomm
