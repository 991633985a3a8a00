// A whole expert layer for a few tokens, in one cooperative kernel.
//
//   out[i][t] = residual[i][t] + sum_s w[i][t][s] * D_e (silu(G_e x) * (U_e x)),   e = idx[i][t][s]
//
// for every token t of every rank i; expert e's matrices (G and U stacked in w_up, D in w_down) lie on
// rank e / (E/p). What the dispatch, the experts and the combine do for many tokens in turn is done here
// without moving a row: few tokens are read where they lie. Phases, with a grid barrier between them:
//   0  every CTA sorts the assignments (token, slot) by expert in its shared memory; no CTA waits for
//      another (redundant, but shorter than a barrier);
//   1  per (picked expert, 8 rows of G and of U, up to 32 of its assignments): both products, then
//      h = silu(g) u. A warp's 16-row tile holds G's rows in its upper half and U's in its lower half,
//      so that one lane's accumulators hold g and u of the same element. The second product's instruction
//      takes bf16; h goes into it in two parts, 16 bits of it. In one part its rounding would show: the error of
//      a layer without a residual grew from the output's rounding alone, 1.66e-3, to 2.37e-3;
//   2  per (picked expert, 16 rows of D, up to 32 assignments): y = D h, fp32;
//   3  per (token, columns): the weighted sum over slots in slot order and the residual, each product and
//      sum rounded to fp32 as in the combine, rounded once.
// The warp-level product and what bounds it are in wprod.cuh. Measured on B200, 4-bit weights of 4096 x 2048: 14 picked
// experts with one assignment each 82 us (the bytes take 29 at the copy rate), 64 of them with 256 assignments 275 us,
// 3.0 TB/s (127); with h in one part 76 and 262. bf16 in moe_tensor.cu and at the rule below; rows that are not whole
// 16-byte units are loaded by element: 16 experts of 1001 x 713 with 33 each 256 us, 45 for 1000 x 712.
#include <algorithm>
#include <type_traits>

#include "moe_layer.cuh"
#include "wprod.cuh"

namespace simcomm {

constexpr int kLayTokens = 32;  // assignments of an expert that one unit covers

// The units of phase 1 (UP) or 2: (picked expert, block of row tiles, up to 32 of its assignments). A warp's
// two row tiles hold rows f..f+7 of G in their upper and of U in their lower halves (UP), or 32 rows of D.
constexpr int kLayTiles = 2;

template <int WK, bool VEC, bool UP> struct LayerJob {
    static constexpr int kWK = WK, kMT = kLayTiles;
    static constexpr bool kVecW = WTraits<WK>::kQ4 || VEC, kVecX = VEC;
    static constexpr int kParts = UP ? 1 : kLayParts;
    static constexpr int kTile = (UP ? 8 : 16) * kMT;  // rows of the output in a group of row tiles
    const MoeLayerArgs& a;
    const LayerLists& l;
    int nact;
    int K, segments, shift, chunk_shift, rows_all, blocks;
    ptrdiff_t part;

    __device__ __forceinline__ LayerJob(const MoeLayerArgs& a_, const LayerLists& l_, int nact_)
        : a(a_), l(l_), nact(nact_), K(UP ? a_.H : a_.F), segments(1), shift(UP ? a_.shift_up : a_.shift_down),
          chunk_shift(a_.chunk_shift), rows_all(UP ? a_.F : a_.H), blocks(UP ? a_.blocks_up : a_.blocks_down), part(a_.h_part) {}

    __device__ __forceinline__ int split_shift(int) const { return shift; }
    __device__ __forceinline__ int units() const { return l.act_tile[nact] * blocks; }
    struct At { int e, row0, first, count; };
    __device__ __forceinline__ At at(int u) const {
        int lo = 0, hi = nact - 1;  // the last picked expert whose units start at or before u
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (l.act_tile[mid] * blocks <= u) lo = mid;
            else hi = mid - 1;
        }
        const int tiles = l.act_tile[lo + 1] - l.act_tile[lo], rel = u - l.act_tile[lo] * blocks;
        At x;
        x.e = l.act[lo];
        x.row0 = rel / tiles * (kProdWarps >> shift) * kTile;
        x.first = l.act_start[lo] + rel % tiles * kLayTokens;
        x.count = min(kLayTokens, l.act_start[lo + 1] - x.first);
        return x;
    }
    // Row g of the upper (i = 0) or lower half of the m-th row tile; rows past the end: the last one.
    __device__ __forceinline__ size_t row_at(const At& x, int tile, int m, int i, int g) const {
        const int r = min(x.row0 + tile * kTile + (UP ? m * 8 : m * 16 + i * 8) + g, rows_all - 1);
        return size_t(x.e % a.E_loc) * (UP ? 2 * a.F : a.H) + r + (UP ? size_t(i) * a.F : 0);
    }
    __device__ __forceinline__ void rows(int u, int, int tile, int g, const char* (&w)[kMT][2]) const {
        const At x = at(u);
        const char* base = UP ? a.up[x.e / a.E_loc] : a.down[x.e / a.E_loc];
        const size_t row_bytes = WTraits<WK>::kQ4 ? size_t(K) / 2 : size_t(K) * 2;
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) w[m][i] = base + row_at(x, tile, m, i, g) * row_bytes;
    }
    __device__ __forceinline__ void scales(int u, int, int tile, int g, int t, const uint16_t* (&s)[(kMT + 1) / 2]) const {
        const At x = at(u);
        s[0] = (UP ? a.up_scale[x.e / a.E_loc] : a.down_scale[x.e / a.E_loc]) +
               row_at(x, tile, t / 2, t % 2, g) * (size_t(K) >> a.group_shift);
    }
    __device__ __forceinline__ const uint16_t* token(int u, int, int n) const {
        const At x = at(u);
        if (n >= x.count) return nullptr;
        if constexpr (UP) {
            const int tok = l.list[x.first + n] / a.k;
            return a.x[a.rank0 + tok / int(a.T)] + size_t(tok % int(a.T)) * a.H;
        } else {
            return a.h + size_t(l.list[x.first + n]) * a.h_stride;
        }
    }
};

// Runs f with the number of 8-token tiles that a count of assignments needs.
template <typename F> __device__ __forceinline__ bool with_tiles(int count, F f) {
    if (count <= 8) return f(std::integral_constant<int, 1>());
    if (count <= 16) return f(std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 4>());
}

template <int WK, bool VEC, bool UP>
__device__ __forceinline__ bool layer_phase(const MoeLayerArgs& a, const LayerLists& l, const ProductSmem& s, PanelCount& pc,
                                            int nact) {
    using Job = LayerJob<WK, VEC, UP>;
    const Job job(a, l, nact);
    const int units = job.units();
    if (threadIdx.x >= kProdWarps * 32) {
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x)
            ok = with_tiles(job.at(u).count, [&](auto nt) {
                return copy_tokens<decltype(nt)::value, Job::kParts>(job, a.ctl, a.timeout_ns, s, pc, u);
            });
        land_panels(a.ctl, s, pc);
        return ok;
    }
    Multiplier<Job> mul(job, s, blockIdx.x, units, gridDim.x);
    if (int(blockIdx.x) == a.fault_cta && threadIdx.x < 32) mul.give_up();
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const typename Job::At x = job.at(u);
        with_tiles(x.count, [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            float acc[kLayTiles][NT][4];
            mul.template unit<NT, Job::kParts>(a.ctl, a.timeout_ns, pc, u, acc);
            finish_unit<UP, kLayTiles, NT>(s, 1 << job.shift, acc, [&](int tile, int r, int c, float v, float v2) {
                const int row = x.row0 + tile * Job::kTile + (UP ? r / 16 * 8 + r % 8 : r);
                if (row >= job.rows_all || c >= x.count || !mul.live) return;
                const int asg = l.list[x.first + c];
                if constexpr (UP) store_h(a, asg, row, silu_mul(v, v2));
                else a.y[size_t(asg) * a.H + row] = v;
            });
            return true;
        });
    }
    mul.drain(a.ctl);
    return mul.live;
}

template <int WK, bool VEC>
__global__ void __launch_bounds__(kProdThreads, 1) k_moe_layer(const __grid_constant__ MoeLayerArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    __shared__ int s_fail;
    if (threadIdx.x == 0) s_fail = status_failed(a.ctl);
    __syncthreads();
    if (s_fail) return;
    const LayerLists l = layer_lists(a, s_raw + product_smem<kLayTiles, kLayParts>());
    const ProductSmem s = product_layout<kLayTiles, kLayParts>(s_raw);
    if (threadIdx.x == 0) init_panels(s);
    const int nact = sort_assignments<kProdThreads>(a, l, kLayTokens);
    if (nact < 0) return;
    PanelCount pc;
    bool ok = layer_phase<WK, VEC, true>(a, l, s, pc, nact);
    if (!layer_barrier(a, 1, ok)) return;
    if constexpr (VEC) {  // h was written by ordinary stores and is read by bulk copies
        asm volatile("fence.proxy.async;" ::: "memory");
    }
    ok = layer_phase<WK, VEC, false>(a, l, s, pc, nact);
    if (!layer_barrier(a, 2, ok)) return;
    weighted_sum<kProdThreads>(a);
    __syncthreads();
    if (threadIdx.x == 0) leave_tasks(&a.st->layer_ctr, &a.st->layer_done);
}

template <int WK, bool VEC> static cudaError_t launch_layer(MoeLayerArgs& a, int num_sms, cudaStream_t s) {
    auto* kernel = k_moe_layer<WK, VEC>;
    const size_t smem = product_smem<kLayTiles, kLayParts>() + layer_lists_bytes(a.E, a.A);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kProdThreads, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorNotSupported;
    const size_t resident = size_t(num_sms) * per_sm;
    const size_t picked = size_t(std::min(a.E, a.A)) + size_t(a.A) / kLayTokens;  // at most this many token tiles
    // Warps of a CTA on one row tile: more, while the tiles do not fill the GPU's warps. Measured on B200 for 16 picked
    // experts of 4096 x 2048 in 4 bits: 79 us so, 92 with twice as many warps to a tile.
    auto plan = [&](size_t tiles, int K, int* shift, int* blocks) {
        const int stages = K / WTraits<WK>::kStageK;
        int sh = 0;
        while ((1 << sh) < max_splits<WK, kLayTokens / 8>() && (2 << sh) <= stages && (picked * tiles << sh) < resident * kProdWarps)
            ++sh;
        *shift = sh;
        const size_t per = kProdWarps >> sh;
        *blocks = int((tiles + per - 1) / per);
    };
    plan((size_t(a.F) + 8 * kLayTiles - 1) / (8 * kLayTiles), a.H, &a.shift_up, &a.blocks_up);
    plan((size_t(a.H) + 16 * kLayTiles - 1) / (16 * kLayTiles), a.F, &a.shift_down, &a.blocks_down);
    const size_t units = picked * size_t(std::max(a.blocks_up, a.blocks_down));
    dim3 grid(unsigned(std::max<size_t>(1, std::min(resident, units)))), block(kProdThreads);
    void* args[] = {&a};
    e = cudaLaunchCooperativeKernel(reinterpret_cast<void*>(kernel), grid, block, args, smem, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// The kernel on the fifth-generation tensor cores needs bf16 weights and rows of 16-byte units. By itself it is
// taken where an expert gets 24 assignments or more, which the streamed products read the weights again for (32 to a
// unit) and multiply at the older instructions' rate; from 12 on where units of 128 rows fill half a round of the SMs in
// both products; and with fewer where they fill one and a half: few units are slow, for their stages of 64 k's wait for
// one another. Measured on B200, us streamed and tensor, by picked experts of H x F and assignments each: 8 of 1024 x
// 1024 with 16 34 and 35, with 24 38 and 39, with 32 56 and 39; 16 of 1000 x 712 with 8 37 and 35, with 12 45 and 38,
// with 32 62 and 47; 8 of 4096 x 2048 with 8 92 and 90, with 12 116 and 98, with 32 191 and 110; 8 of 1024 x 512 with 16
// 27 and 31, 4 of 2048 x 4096 with 16 77 and 80; with one assignment each, 2 of 4096 x 2048 21 and 54, 14 of them 152
// and 144, 8 of 4096 x 14336 492 and 446, 4 of them 222 and 233; 64 of 1024 x 1024 with 2 87 and 87.
static bool layer_takes_tensor(const MoeLayerArgs& a, int num_sms) {
    if (a.tensor == 0 || a.weight_kind != COLL_WEIGHT_BF16 || !a.vec || !layer_tensor_fits(a)) return false;
    const int experts = std::min(a.E, a.A), units = experts * ((std::min(a.H, a.F) + 127) / 128);
    return a.tensor == 1 || a.A >= 24 * experts || (a.A >= 12 * experts && units * 2 >= num_sms) || units * 2 >= num_sms * 3;
}

cudaError_t launch_moe_layer(const MoeLayerArgs& args, int num_sms, cudaStream_t s) {
    MoeLayerArgs a = args;
    if (layer_takes_tensor(a, num_sms)) return launch_layer_tensor(a, num_sms, s);
    if (a.weight_kind == 0)
        return a.vec ? launch_layer<W_BF16, true>(a, num_sms, s) : launch_layer<W_BF16, false>(a, num_sms, s);
    const int group = 1 << a.group_shift;
    a.chunk_shift = 0;
    while ((128 << a.chunk_shift) < group) ++a.chunk_shift;
    if (group >= 128)
        return a.vec ? launch_layer<W_Q4X4, true>(a, num_sms, s) : launch_layer<W_Q4X4, false>(a, num_sms, s);
    if (group == 64)
        return a.vec ? launch_layer<W_Q4X2, true>(a, num_sms, s) : launch_layer<W_Q4X2, false>(a, num_sms, s);
    return a.vec ? launch_layer<W_Q4X1, true>(a, num_sms, s) : launch_layer<W_Q4X1, false>(a, num_sms, s);
}

}  // namespace simcomm
