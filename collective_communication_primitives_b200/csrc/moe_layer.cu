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
//      so that one lane's accumulators hold g and u of the same element. h is rounded to bf16, the type
//      that the second product's instruction takes (its relative error of 2^-9 a term averages out in a
//      sum of F terms to less than the rounding of the output);
//   2  per (picked expert, 16 rows of D, up to 32 assignments): y = D h, fp32;
//   3  per (token, columns): the weighted sum over slots in slot order and the residual, each product and
//      sum rounded to fp32 as in the combine, rounded once.
// Bound by the bytes of the picked experts' weights; the warp-level product is in wprod.cuh.
#include <algorithm>

#include "wprod.cuh"

namespace simcomm {

constexpr int kLayWarps = 8;
constexpr int kLayThreads = kLayWarps * 32;
constexpr int kLayTokens = 32;  // assignments of an expert that one unit covers

__device__ __forceinline__ bool layer_barrier(const MoeLayerArgs& a, uint32_t k) {
    __shared__ int s_ok;
    __syncthreads();
    if (threadIdx.x == 0) {
        red_release_add_gpu(&a.st->layer_ctr, 1u);
        const uint32_t want = k * gridDim.x;
        s_ok = wait_counter(a.ctl, &a.st->layer_ctr, want, a.timeout_ns) && !status_failed(a.ctl);
    }
    __syncthreads();
    return s_ok != 0;
}

struct LayerLists {
    int* offset;      // [E] while counting: count, then next free place of the expert in list
    int* act_start;   // [nact + 1] first place of the i-th picked expert in list
    int* act_tile;    // [nact + 1] its first token tile
    uint16_t* act;    // [nact] its id
    uint16_t* list;   // [A] assignments, expert by expert
};

__device__ __forceinline__ int warp_incl_sum(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Exclusive prefix over the CTA of three counts per thread; their totals in tot.
__device__ __forceinline__ void cta_prefix3(int (&v)[3], int (&tot)[3]) {
    __shared__ int s_w[3][kLayWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int incl[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        incl[q] = warp_incl_sum(v[q], lane);
        if (lane == 31) s_w[q][warp] = incl[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        int before = 0;
        tot[q] = 0;
        for (int w = 0; w < kLayWarps; ++w) {
            if (w < warp) before += s_w[q][w];
            tot[q] += s_w[q][w];
        }
        v[q] = before + incl[q] - v[q];
    }
    __syncthreads();
}

// Phase 0. Returns the number of picked experts, or -1 after an expert id out of range.
__device__ __forceinline__ int sort_assignments(const MoeLayerArgs& a, const LayerLists& l) {
    __shared__ int s_bad;
    const int per = int(a.T) * a.k;
    for (int e = threadIdx.x; e < a.E; e += kLayThreads) l.offset[e] = 0;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.A; i += kLayThreads) {
        const int e = a.idx[a.rank0 + i / per][i % per];
        if (e < 0 || e >= a.E) s_bad = 1;
        else atomicAdd(&l.offset[e], 1);
    }
    __syncthreads();
    if (s_bad) {
        if (threadIdx.x == 0) raise_status(a.ctl, COLL_ERR_INVALID_ARG);
        return -1;
    }
    const int share = (a.E + kLayThreads - 1) / kLayThreads;
    const int e0 = min(a.E, int(threadIdx.x) * share), e1 = min(a.E, e0 + share);
    int v[3] = {0, 0, 0}, tot[3];
    for (int e = e0; e < e1; ++e) {
        const int c = l.offset[e];
        v[0] += c > 0;
        v[1] += c;
        v[2] += (c + kLayTokens - 1) / kLayTokens;
    }
    cta_prefix3(v, tot);
    for (int e = e0; e < e1; ++e) {
        const int c = l.offset[e];
        l.offset[e] = v[1];
        if (c == 0) continue;
        l.act[v[0]] = uint16_t(e);
        l.act_start[v[0]] = v[1];
        l.act_tile[v[0]] = v[2];
        v[0] += 1;
        v[1] += c;
        v[2] += (c + kLayTokens - 1) / kLayTokens;
    }
    if (threadIdx.x == 0) {
        l.act_start[tot[0]] = tot[1];
        l.act_tile[tot[0]] = tot[2];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.A; i += kLayThreads)
        l.list[atomicAdd(&l.offset[a.idx[a.rank0 + i / per][i % per]], 1)] = uint16_t(i);
    __syncthreads();
    // The atomics leave an expert's assignments in an order that differs from CTA to CTA. That does not
    // matter inside one token tile (an assignment's result does not depend on its column), but every CTA
    // must cut an expert's assignments into the same tiles: those with more than one are put in order, a
    // warp per expert, by a bitmap of the assignments.
    __shared__ uint32_t s_bits[kLayWarps][kLayerMaxAssignments / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* bits = s_bits[warp];
    constexpr int kWords = kLayerMaxAssignments / 32 / 32;  // bitmap words per lane
    for (int q = warp; q < tot[0]; q += kLayWarps) {
        const int start = l.act_start[q], n = l.act_start[q + 1] - start;
        if (n <= kLayTokens) continue;
        for (int w = lane; w < kLayerMaxAssignments / 32; w += 32) bits[w] = 0u;
        __syncwarp();
        for (int i = lane; i < n; i += 32) atomicOr(&bits[l.list[start + i] >> 5], 1u << (l.list[start + i] & 31));
        __syncwarp();
        int mine = 0;
        for (int w = 0; w < kWords; ++w) mine += __popc(bits[lane * kWords + w]);
        int at = start + warp_incl_sum(mine, lane) - mine;
        for (int w = 0; w < kWords; ++w)
            for (uint32_t b = bits[lane * kWords + w]; b; b &= b - 1)
                l.list[at++] = uint16_t((lane * kWords + w) * 32 + __ffs(b) - 1);
        __syncwarp();
    }
    __syncthreads();
    return tot[0];
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// One unit of phase 1 (UP) or 2: up to 8 NT assignments of one expert against the CTA's row tiles.
template <int WK, bool VEC, int NT, bool UP>
__device__ __forceinline__ void layer_unit(const MoeLayerArgs& a, const LayerLists& l, float* s_red, int e, int first,
                                           int count, int blk) {
    using W = WTraits<WK>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int splits = UP ? a.splits_up : a.splits_down, per = kLayWarps / splits, split = warp % splits;
    const int K = UP ? a.H : a.F, rows = UP ? a.F : a.H, tile_rows = UP ? 8 : 16;
    const int rank = e / a.E_loc, el = e % a.E_loc;
    const int row0 = (blk * per + warp / splits) * tile_rows;
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    if (row0 < rows) {
        const int chunks = (K + W::kChunk - 1) / W::kChunk;
        const int lo = int((long long)chunks * split / splits), hi = int((long long)chunks * (split + 1) / splits);
        const size_t wrow = W::kQ4 ? size_t(K) / 2 : size_t(K) * 2;
        const size_t base = size_t(el) * (UP ? 2 * a.F : a.H);
        const size_t r0 = base + row0 + g, r1 = UP ? r0 + a.F : r0 + 8;
        const bool in0 = row0 + g < rows, in1 = UP ? in0 : row0 + g + 8 < rows;
        const char* w = UP ? a.up[rank] : a.down[rank];
        LaneRows lr;
        lr.w0 = in0 ? w + r0 * wrow : nullptr;
        lr.w1 = in1 ? w + r1 * wrow : nullptr;
        lr.s0 = lr.s1 = nullptr;
        if constexpr (W::kQ4) {
            const uint16_t* sc = UP ? a.up_scale[rank] : a.down_scale[rank];
            const size_t srow = size_t(K) >> a.group_shift;
            lr.s0 = sc + r0 * srow;
            lr.s1 = sc + r1 * srow;
        }
        const uint16_t* x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int c = n * 8 + g;
            x[n] = nullptr;
            if (c < count) {
                const int asg = l.list[first + c];
                if constexpr (UP) {
                    const int tok = asg / a.k;
                    x[n] = a.x[a.rank0 + tok / int(a.T)] + size_t(tok % int(a.T)) * a.H;
                } else {
                    x[n] = a.h + size_t(asg) * a.h_stride;
                }
            }
        }
        warp_product<WK, VEC, NT>(acc, lr, x, lo, hi, K, a.chunk_shift, t);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_red[(warp * 4 * NT + 4 * n + i) * 32 + lane] = acc[n][i];
    __syncthreads();
    for (int x = threadIdx.x; x < per * tile_rows * 8 * NT; x += kLayThreads) {
        const int r = x % tile_rows, c = (x / tile_rows) % (8 * NT), q = x / (tile_rows * 8 * NT);
        const int row = (blk * per + q) * tile_rows + r;
        if (row >= rows || c >= count) continue;
        const int asg = l.list[first + c];
        const int ln = (r % 8) * 4 + (c % 8) / 2, reg = 4 * (c / 8) + (c & 1) + (r / 8) * 2;
        float v = 0.0f, v2 = 0.0f;
        for (int s = 0; s < splits; ++s) {
            const float* red = s_red + (q * splits + s) * 4 * NT * 32 + ln;
            v += red[reg * 32];
            if (UP) v2 += red[(reg + 2) * 32];
        }
        if constexpr (UP) a.h[size_t(asg) * a.h_stride + row] = float_to_bf16_bits(silu_mul(v, v2));
        else a.y[size_t(asg) * a.H + row] = v;
    }
    __syncthreads();  // the next unit writes s_red
}

template <int WK, bool VEC, bool UP>
__device__ __forceinline__ void layer_phase(const MoeLayerArgs& a, const LayerLists& l, float* s_red, int nact) {
    const int blocks = UP ? a.blocks_up : a.blocks_down;
    const int units = l.act_tile[nact] * blocks;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        int lo = 0, hi = nact - 1;  // the last picked expert whose units start at or before u
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (l.act_tile[mid] * blocks <= u) lo = mid;
            else hi = mid - 1;
        }
        const int tiles = l.act_tile[lo + 1] - l.act_tile[lo];
        const int rel = u - l.act_tile[lo] * blocks;
        const int blk = rel / tiles, tile = rel % tiles;
        const int first = l.act_start[lo] + tile * kLayTokens;
        const int count = min(kLayTokens, l.act_start[lo + 1] - first);
        const int e = l.act[lo];
        if (count <= 8) layer_unit<WK, VEC, 1, UP>(a, l, s_red, e, first, count, blk);
        else if (count <= 16) layer_unit<WK, VEC, 2, UP>(a, l, s_red, e, first, count, blk);
        else layer_unit<WK, VEC, 4, UP>(a, l, s_red, e, first, count, blk);
    }
}

template <int WK, bool VEC>
__global__ void __launch_bounds__(kLayThreads, 2) k_moe_layer(const __grid_constant__ MoeLayerArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    __shared__ float s_red[kLayWarps * 4 * (kLayTokens / 8) * 32];
    __shared__ int s_fail;
    if (threadIdx.x == 0) s_fail = status_failed(a.ctl);
    __syncthreads();
    if (s_fail) return;
    const int most = min(a.E, a.A);
    LayerLists l;
    l.offset = reinterpret_cast<int*>(s_raw);
    l.act_start = l.offset + a.E;
    l.act_tile = l.act_start + most + 1;
    l.act = reinterpret_cast<uint16_t*>(l.act_tile + most + 1);
    l.list = l.act + most;
    const int nact = sort_assignments(a, l);
    if (nact < 0) return;
    layer_phase<WK, VEC, true>(a, l, s_red, nact);
    if (!layer_barrier(a, 1)) return;
    layer_phase<WK, VEC, false>(a, l, s_red, nact);
    if (!layer_barrier(a, 2)) return;
    // the weighted sum: a thread per token and column
    const int tokens = a.A / a.k;
    const size_t total = size_t(tokens) * a.H;
    for (size_t i = size_t(blockIdx.x) * kLayThreads + threadIdx.x; i < total; i += size_t(gridDim.x) * kLayThreads) {
        const int tok = int(i / a.H), col = int(i % a.H);
        const int rank = a.rank0 + tok / int(a.T);
        const size_t at = size_t(tok % int(a.T)) * a.H + col;
        const float* w = a.weight[rank] + size_t(tok % int(a.T)) * a.k;
        const float* y = a.y + size_t(tok) * a.k * a.H + col;
        float v = a.has_res ? bf16_bits_to_float(a.res[rank][at]) : 0.0f;
        for (int s = 0; s < a.k; ++s) {
            const float term = w[s] * y[size_t(s) * a.H];
            v = (s == 0 && !a.has_res) ? term : v + term;
        }
        a.out[rank][at] = float_to_bf16_bits(v);
    }
    __syncthreads();
    if (threadIdx.x == 0) leave_tasks(&a.st->layer_ctr, &a.st->layer_done);
}

size_t moe_layer_lists_bytes(int E, int A) {
    const size_t most = size_t(std::min(E, A));
    return size_t(E) * 4 + (most + 1) * 8 + most * 2 + size_t(A) * 2;
}

template <int WK, bool VEC> static cudaError_t launch_layer(MoeLayerArgs& a, int num_sms, cudaStream_t s) {
    auto* kernel = k_moe_layer<WK, VEC>;
    const size_t smem = moe_layer_lists_bytes(a.E, a.A);
    cudaError_t e = cudaSuccess;
    if (smem > 32 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kLayThreads, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorNotSupported;
    const size_t resident = size_t(num_sms) * per_sm;
    const size_t picked = size_t(std::min(a.E, a.A)) + size_t(a.A) / kLayTokens;  // at most this many token tiles
    // warps of a CTA on one row tile: more, the fewer tiles there are to fill the GPU with
    auto plan = [&](size_t tiles, int* splits, int* blocks) {
        int sp = 1;
        while (sp < kLayWarps && picked * tiles * sp < resident * 8 * kLayWarps) sp *= 2;
        *splits = sp;
        const size_t per = kLayWarps / sp;
        *blocks = int((tiles + per - 1) / per);
    };
    plan((size_t(a.F) + 7) / 8, &a.splits_up, &a.blocks_up);
    plan((size_t(a.H) + 15) / 16, &a.splits_down, &a.blocks_down);
    const size_t units = picked * size_t(std::max(a.blocks_up, a.blocks_down));
    dim3 grid(unsigned(std::max<size_t>(1, std::min(resident, units)))), block(kLayThreads);
    void* args[] = {&a};
    e = cudaLaunchCooperativeKernel(reinterpret_cast<void*>(kernel), grid, block, args, smem, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_moe_layer(const MoeLayerArgs& args, int num_sms, cudaStream_t s) {
    MoeLayerArgs a = args;
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
