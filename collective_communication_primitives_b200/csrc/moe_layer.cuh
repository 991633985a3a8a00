// What the expert layer's kernels share: the order of the assignments, the grid barrier, the weighted sum.
#pragma once

#include "common.cuh"

namespace simcomm {

__device__ __forceinline__ bool layer_barrier(const MoeLayerArgs& a, uint32_t k, bool ok) {
    __shared__ int s_ok;
    if (!__syncthreads_and(ok)) return false;  // a wait ran out: the status is set
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
template <int THREADS> __device__ __forceinline__ void cta_prefix3(int (&v)[3], int (&tot)[3]) {
    constexpr int kWarps = THREADS / 32;
    __shared__ int s_w[3][kWarps];
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
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += s_w[q][w];
            tot[q] += s_w[q][w];
        }
        v[q] = before + incl[q] - v[q];
    }
    __syncthreads();
}

// Phase 0. Returns the number of picked experts, or -1 after an expert id out of range. `tile`: assignments of an
// expert that one unit covers.
template <int THREADS>
__device__ __forceinline__ int sort_assignments(const MoeLayerArgs& a, const LayerLists& l, int tile) {
    __shared__ int s_bad;
    const int per = int(a.T) * a.k;
    for (int e = threadIdx.x; e < a.E; e += THREADS) l.offset[e] = 0;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    // this thread's ids, all loads in flight together
    constexpr int kMine = (kLayerMaxAssignments + THREADS - 1) / THREADS;
    int ids[kMine];
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        const int i = q * THREADS + threadIdx.x;
        ids[q] = i < a.A ? __ldg(a.idx[a.rank0 + i / per] + i % per) : -1;
    }
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        if (q * THREADS + int(threadIdx.x) >= a.A) break;
        if (ids[q] < 0 || ids[q] >= a.E) s_bad = 1;
        else atomicAdd(&l.offset[ids[q]], 1);
    }
    __syncthreads();
    if (s_bad) {
        if (threadIdx.x == 0) raise_status(a.ctl, COLL_ERR_INVALID_ARG);
        return -1;
    }
    const int share = (a.E + THREADS - 1) / THREADS;
    const int e0 = min(a.E, int(threadIdx.x) * share), e1 = min(a.E, e0 + share);
    int v[3] = {0, 0, 0}, tot[3];
    for (int e = e0; e < e1; ++e) {
        const int c = l.offset[e];
        v[0] += c > 0;
        v[1] += c;
        v[2] += (c + tile - 1) / tile;
    }
    cta_prefix3<THREADS>(v, tot);
    for (int e = e0; e < e1; ++e) {
        const int c = l.offset[e];
        l.offset[e] = v[1];
        if (c == 0) continue;
        l.act[v[0]] = uint16_t(e);
        l.act_start[v[0]] = v[1];
        l.act_tile[v[0]] = v[2];
        v[0] += 1;
        v[1] += c;
        v[2] += (c + tile - 1) / tile;
    }
    if (threadIdx.x == 0) {
        l.act_start[tot[0]] = tot[1];
        l.act_tile[tot[0]] = tot[2];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        const int i = q * THREADS + threadIdx.x;
        if (i >= a.A) break;
        l.list[atomicAdd(&l.offset[ids[q]], 1)] = uint16_t(i);
    }
    __syncthreads();
    // The atomics leave an expert's assignments in an order that differs from CTA to CTA. That does not
    // matter inside one token tile (an assignment's result does not depend on its column), but every CTA
    // must cut an expert's assignments into the same tiles: those with more than one are put in order, a
    // warp per expert, by a bitmap of the assignments.
    __shared__ uint32_t s_bits[THREADS / 32][kLayerMaxAssignments / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* bits = s_bits[warp];
    constexpr int kWords = kLayerMaxAssignments / 32 / 32;  // bitmap words per lane
    for (int q = warp; q < tot[0]; q += THREADS / 32) {
        const int start = l.act_start[q], n = l.act_start[q + 1] - start;
        if (n <= tile) continue;
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

// h of an assignment in two bf16 parts: its rounding, and what that left out (none of an infinity or NaN).
constexpr int kLayParts = 2;
__device__ __forceinline__ void store_h(const MoeLayerArgs& a, int asg, int row, float h) {
    uint16_t* to = a.h + size_t(asg) * a.h_stride + row;
    const uint16_t high = float_to_bf16_bits(h);
    const float rest = h - bf16_bits_to_float(high);
    to[0] = high;
    to[a.h_part] = fabsf(rest) < INFINITY ? float_to_bf16_bits(rest) : uint16_t(0);
}

// Phase 3: the weighted sum, a thread per token and N columns. y was written by other CTAs before the barrier.
template <int THREADS, int N> __device__ __forceinline__ void weighted_sum_of(const MoeLayerArgs& a) {
    const int tokens = a.A / a.k, pieces = a.H / N;
    const size_t total = size_t(tokens) * pieces;
    for (size_t i = size_t(blockIdx.x) * THREADS + threadIdx.x; i < total; i += size_t(gridDim.x) * THREADS) {
        const int tok = int(i / pieces), col = int(i % pieces) * N;
        const int rank = a.rank0 + tok / int(a.T), t = tok % int(a.T);
        const size_t at = size_t(t) * a.H + col;
        const float* w = a.weight[rank] + size_t(t) * a.k;
        const float* y = a.y + size_t(tok) * a.k * a.H + col;
        float v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = a.has_res ? bf16_bits_to_float(a.res[rank][at + j]) : 0.0f;
#pragma unroll 4
        for (int s = 0; s < a.k; ++s) {
            float x[N];
            if constexpr (N == 4) {
                const float4 q = *reinterpret_cast<const float4*>(y + size_t(s) * a.H);
                x[0] = q.x; x[1] = q.y; x[2] = q.z; x[3] = q.w;
            } else {
                x[0] = y[size_t(s) * a.H];
            }
            const float ws = w[s];
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = (s == 0 && !a.has_res) ? ws * x[j] : v[j] + ws * x[j];
        }
#pragma unroll
        for (int j = 0; j < N; ++j) a.out[rank][at + j] = float_to_bf16_bits(v[j]);
    }
}
template <int THREADS> __device__ __forceinline__ void weighted_sum(const MoeLayerArgs& a) {
    if (a.H % 4 == 0) weighted_sum_of<THREADS, 4>(a);  // y's rows are then 16-byte aligned
    else weighted_sum_of<THREADS, 1>(a);
}

// The lists' place in `smem`, layer_lists_bytes long.
__device__ __forceinline__ LayerLists layer_lists(const MoeLayerArgs& a, unsigned char* smem) {
    const int most = min(a.E, a.A);
    LayerLists l;
    l.offset = reinterpret_cast<int*>(smem);
    l.act_start = l.offset + a.E;
    l.act_tile = l.act_start + most + 1;
    l.act = reinterpret_cast<uint16_t*>(l.act_tile + most + 1);
    l.list = l.act + most;
    return l;
}
inline size_t layer_lists_bytes(int E, int A) {
    const size_t most = size_t(E < A ? E : A);
    return size_t(E) * 4 + (most + 1) * 8 + most * 2 + size_t(A) * 2;
}

// Programs launch_moe_layer chooses between.
bool layer_tensor_fits(const MoeLayerArgs& a);  // its shared memory holds the lists too
cudaError_t launch_layer_tensor(MoeLayerArgs a, int num_sms, cudaStream_t s);

}  // namespace simcomm
