// The expert layer (moe_layer.cu) for bf16 weights and many assignments an expert: the same phases, the two
// products on the fifth-generation tensor cores.
//
//   D[r][n] = sum_k W[r][k] X[n][k]:  tcgen05.mma, 128 weight rows x 16..128 assignments, k by 64
//
// Weights are the 128-row operand: with few tokens they are the long side, and every weight then passes
// through an SM once per 128 assignments of its expert. Both operands are K-major in shared memory in the
// 128-byte swizzle (a row's 64 k's are 128 bytes, whose 16-byte pieces are permuted by the row's low bits),
// accumulators are in tensor memory. One CTA per SM, its warps in three roles that run on from unit to unit:
//   warps 5-8  copy the operands' rows ahead into a ring of stages (cp.async, 16 bytes per thread). The rows
//              are taken from where they lie, by pointer: weight rows in the order that the epilogue wants,
//              token rows through the list of assignments, so nothing is gathered beforehand;
//   warp 4     one thread issues the matrix instructions of a stage, whose completion frees the stage;
//   warps 0-3  read a finished accumulator (two alternate) and write the results.
// In phase 2 a stage holds both parts of the tokens' values, operands of two instructions into the same accumulator.
// In phase 1 a group of 32 accumulator lanes holds 16 rows of G and the same 16 of U, so that silu(g) u needs one
// exchange between lanes of a warp. A unit is M row tiles of 128: with two, the tokens' rows are staged
// half as often. Bound by the weights' bytes while an expert has fewer than about 100 assignments. Measured on B200
// with experts of 4096 x 2048: 64 of them with 64 assignments each 607 us, 5.3 TB/s, 0.83 of the copy rate (with h in
// one part 572); 14 with one each 143 us, 5.0 TB/s (the two products' ends weigh more). Of 50 us for 16 of 1000 x 712 with
// 33 each, caches cold, the order takes 3.5, the first product 24, the first barrier 4 to 6, the second product with
// its barrier 16, the sum 2.6.
#include <algorithm>

#include "moe_layer.cuh"

namespace simcomm {

constexpr int kTcEpilogue = 4, kTcCopy = 4;                       // warps
constexpr int kTcThreads = (kTcEpilogue + 1 + kTcCopy) * 32;
constexpr int kTcTokens = 128;                                    // assignments of a unit
constexpr int kTcK = 64;                                          // k's of a stage
constexpr int kTcTileBytes = 128 * kTcK * 2;                      // 128 rows of a stage
constexpr int kTcTiles = 2;                                       // row tiles of a unit, at most
constexpr int kTcStages = 16;                                     // stages, at most
constexpr int kTcRing = 192 * 1024;                               // bytes of the ring of stages, at least
constexpr uint64_t kTcIdleNs = 1000000000ull;                     // longest wait for instructions in flight before leaving

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}
// One lane of the warp, in a form that tells the compiler so: the instructions' operands stay in uniform registers.
// (By a test of the lane's number a stage took 0.1 us longer to issue.)
__device__ __forceinline__ bool elected() {
    uint32_t mine;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(mine));
    return mine != 0u;
}
// Shared-memory descriptor of a K-major tile in the 128-byte swizzle: groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t tc_desc(uint32_t smem) {
    return uint64_t((smem & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
           (uint64_t(2) << 61);
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// 16 columns of a lane's row of the accumulator.
__device__ __forceinline__ void tc_load16(float (&v)[16], uint32_t at) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_copy16(uint32_t smem, const void* g, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" :: "r"(smem), "l"(g), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tc_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_u32(bar)) : "memory");
}

// Barriers of a CTA: stages copied and free, one set for each phase, accumulators finished and read, and no instruction
// left in flight (after a wait that ran out).
struct TcBars {
    uint64_t full[2][kTcStages], empty[2][kTcStages], done[2], read[2], idle;
};

// A unit: `span` rows from row0 of an expert's output, assignments [first, first + count). The span is a
// multiple of 16, at most 64 M (UP) or 128 M rows.
template <bool UP> struct TcPhase {
    static constexpr int M = kTcTiles;
    const MoeLayerArgs& a;
    const LayerLists& l;
    int nact, K, rows, span, blocks;
    // A stage: the span's weight rows (128 bytes each), then up to 128 token rows. A last row tile of fewer than
    // 128 rows is read by the matrix instruction as if it were whole: what follows it in the ring gives rows of
    // the accumulator that nobody reads. So small spans have short stages, and many of them.
    int weight_bytes, slot_bytes, stages;
    static constexpr int kTile = UP ? 64 : 128;  // rows of the output in a row tile
    __device__ __forceinline__ TcPhase(const MoeLayerArgs& a_, const LayerLists& l_, int n, int most)
        : a(a_), l(l_), nact(n), K(UP ? a_.H : a_.F), rows(UP ? a_.F : a_.H) {
        // Where whole row tiles would leave CTAs without a unit, the smallest span that still takes one round.
        // With more units than CTAs whole tiles are best, ragged rounds and all: the CTAs of a last, partial round
        // have the memory to themselves. (Measured on 14 picked experts of 4096 x 2048: 142 us with whole tiles in
        // 1.5 rounds, 147 with spans that make two even rounds, 162 and 169 with three and four.)
        // Results do not depend on the span: every unit sums over k from its beginning. (Units that began at different
        // k's, so as not to read the same columns of their rows at the same time, were 1 to 3% faster, but the order of
        // a row's sum then went by which other experts were picked.)
        const int tiles = l.act_tile[nact], grid = int(gridDim.x);
        span = kTile * M;
        while (span > 16 && (rows + span - 17) / (span - 16) * tiles <= grid) span -= 16;
        blocks = (rows + span - 1) / span;
        weight_bytes = span * (UP ? 256 : 128);
        slot_bytes = weight_bytes + token_rows(min(kTcTokens, most)) * 128;
        stages = min(kTcStages, (a.tensor_ring - (weight_bytes % kTcTileBytes ? kTcTileBytes : 0)) / slot_bytes);
    }
    // Rows of a stage for so many assignments: those of one part (an instruction's columns: a multiple of 16), and all.
    static constexpr int kParts = UP ? 1 : kLayParts;
    __device__ __forceinline__ static int part_rows(int count) { return (count + 15) / 16 * 16; }
    __device__ __forceinline__ static int token_rows(int count) { return kParts * part_rows(count); }
    __device__ __forceinline__ int units() const { return l.act_tile[nact] * blocks; }
    __device__ __forceinline__ int row_tiles() const { return (span + kTile - 1) / kTile; }
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
        x.row0 = rel / tiles * span;
        x.first = l.act_start[lo] + rel % tiles * kTcTokens;
        x.count = min(kTcTokens, l.act_start[lo + 1] - x.first);
        return x;
    }
};

// The copying warps' side of a phase.
template <bool UP>
__device__ __forceinline__ bool tc_copy(const TcPhase<UP>& ph, uint32_t smem, TcBars& bars) {
    constexpr int M = kTcTiles;
    const MoeLayerArgs& a = ph.a;
    uint64_t *full = bars.full[UP], *empty = bars.empty[UP];
    const int i = threadIdx.x - (kTcEpilogue + 1) * 32, c = i & 7, r0 = i >> 3;  // this thread's piece and first row
    const uint32_t off = uint32_t(r0 * 128 + ((c ^ (r0 & 7)) << 4));            // rows r0 + 16 j lie 2048 j further
    int slot = 0;
    uint32_t parity = 1u;  // of the wait for a free slot: flips with each turn of the ring
    const int units = ph.units(), kbs = (ph.K + kTcK - 1) / kTcK;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const auto x = ph.at(u);
        const int el = x.e % a.E_loc, rank = x.e / a.E_loc, nb = ph.token_rows(x.count) / 16, part = ph.part_rows(x.count) / 16;
        const char* w[M][8];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                size_t row;  // rows past the end: the last one, whose results are not used
                if constexpr (UP) {
                    const int f = min(x.row0 + m * 64 + (j / 2) * 16 + r0, ph.rows - 1);
                    row = size_t(el) * 2 * a.F + f + (j % 2 ? a.F : 0);
                } else {
                    row = size_t(el) * a.H + min(x.row0 + m * 128 + j * 16 + r0, ph.rows - 1);
                }
                w[m][j] = (UP ? a.up[rank] : a.down[rank]) + (row * ph.K + c * 8) * 2;
            }
        constexpr int kB = TcPhase<UP>::kParts * kTcTokens / 16;
        const char* b[kB];
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            b[j] = nullptr;
            if (j >= nb) continue;
            const bool low = j >= part;  // the second part; rows past the count: the last one
            const int asg = ph.l.list[x.first + min((low ? j - part : j) * 16 + r0, x.count - 1)];
            if constexpr (UP) {
                const int tok = asg / a.k;
                b[j] = reinterpret_cast<const char*>(a.x[a.rank0 + tok / int(a.T)] + size_t(tok % int(a.T)) * a.H + c * 8);
            } else {
                b[j] = reinterpret_cast<const char*>(a.h + size_t(asg) * a.h_stride + (low ? a.h_part : 0) + c * 8);
            }
        }
        for (int kb = 0; kb < kbs; ++kb) {
            if (!mbar_wait_bounded(a.ctl, &empty[slot], parity, a.timeout_ns)) {
                ok = false;
                break;
            }
            const bool in = kb * kTcK + c * 8 < ph.K;
            const size_t at = in ? size_t(kb) * (kTcK * 2) : 0;
            const ptrdiff_t back = in ? 0 : -ptrdiff_t(c) * 16;  // past the end nothing is read; stay in the row
            const uint32_t to = smem + slot * ph.slot_bytes + off, bytes = in ? 16u : 0u;
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int j = 0; j < 8; ++j)  // rows past the span are left as they are: no result of theirs is used
                    if (m * ph.kTile + (UP ? j / 2 : j) * 16 < ph.span)
                        tc_copy16(to + m * kTcTileBytes + j * 2048, w[m][j] + at + back, bytes);
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                if (j >= nb) break;
                tc_copy16(to + ph.weight_bytes + j * 2048, b[j] + at + back, bytes);
            }
            // the barrier hears from this thread when its copies are in; many stages are in flight at a time
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(&full[slot])) : "memory");
            if (++slot == ph.stages) {
                slot = 0;
                parity ^= 1u;
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return ok;
}

// Asks for the first weights of the next phase's first unit before the grid barrier: they do not depend on it.
template <bool UP> __device__ __forceinline__ void tc_prefetch(const TcPhase<UP>& ph) {
    constexpr int kLines = 6;  // of 128 bytes a row
    if (int(blockIdx.x) >= ph.units()) return;
    const MoeLayerArgs& a = ph.a;
    const auto x = ph.at(blockIdx.x);
    const char* w = (UP ? a.up[x.e / a.E_loc] : a.down[x.e / a.E_loc]) +
                    (size_t(x.e % a.E_loc) * (UP ? 2 * a.F : a.H) + x.row0) * ph.K * 2;
    const size_t row_bytes = size_t(ph.K) * 2;
    const int n = min(ph.span, ph.rows - x.row0);
    for (int i = threadIdx.x - (kTcEpilogue + 1) * 32; i < n * kLines; i += kTcCopy * 32) {
        const size_t at = size_t(i % kLines) * 128;
        if (at < row_bytes) asm volatile("prefetch.global.L2 [%0];" :: "l"(w + i / kLines * row_bytes + at));
    }
}

// What the issuing thread does after a wait that ran out: the matrix instructions that it has issued read shared memory
// and write the accumulators, so the CTA stays until they are through.
__device__ __forceinline__ bool tc_quit(const Ctl& ctl, TcBars& bars) {
    tc_commit(&bars.idle);
    mbar_wait_bounded(ctl, &bars.idle, 0u, kTcIdleNs);
    return false;
}

// The issuing thread's side of a phase. acc: accumulators begun.
template <bool UP>
__device__ __forceinline__ bool tc_issue(const TcPhase<UP>& ph, uint32_t smem, TcBars& bars, uint32_t tmem, uint32_t& acc) {
    constexpr int M = kTcTiles;
    const MoeLayerArgs& a = ph.a;
    uint64_t *full = bars.full[UP], *empty = bars.empty[UP];
    int slot = 0;
    uint32_t parity = 0u;
    const int units = ph.units(), kbs = (ph.K + kTcK - 1) / kTcK, tiles = ph.row_tiles();
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++acc) {
        const int part = ph.part_rows(ph.at(u).count);
        // fp32 accumulator, bf16 operands, both K-major, N = part, M = 128
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(part / 8) << 17) | (8u << 24);
        if (!mbar_wait_bounded(a.ctl, &bars.read[acc & 1], (acc / 2 & 1u) ^ 1u, a.timeout_ns)) return tc_quit(a.ctl, bars);
        tc_fence_after();
        const uint32_t d = tmem + (acc & 1) * (M * 128);
        for (int kb = 0; kb < kbs; ++kb) {
            if (!mbar_wait_bounded(a.ctl, &full[slot], parity, a.timeout_ns)) return tc_quit(a.ctl, bars);
            if (int(blockIdx.x) == a.fault_cta && kb == 1) return tc_quit(a.ctl, bars);  // fault injection
            // What the copies wrote is read through another path. The fence stands on this side: a copying thread's
            // would wait for all its copies in flight, 0.7 us a stage.
            fence_proxy_async_smem();
            tc_fence_after();
            const uint32_t at = smem + slot * ph.slot_bytes;
            const uint64_t db = tc_desc(at + ph.weight_bytes);
#pragma unroll
            for (int kk = 0; kk < kTcK / 16; ++kk)  // 16 k's are 32 bytes further in the swizzled rows
#pragma unroll
                for (int m = 0; m < M; ++m)
                    if (m < tiles)
#pragma unroll
                        for (int q = 0; q < ph.kParts; ++q)  // the parts' rows are part * 128 bytes apart
                            tc_mma(d + m * 128, tc_desc(at + m * kTcTileBytes) + kk * 2, db + q * part * 8 + kk * 2, idesc,
                                   uint32_t(kb | kk | q));
            tc_commit(&empty[slot]);
            if (++slot == ph.stages) {
                slot = 0;
                parity ^= 1u;
            }
        }
        tc_commit(&bars.done[acc & 1]);
    }
    return true;
}

// The reading warps' side of a phase.
template <bool UP>
__device__ __forceinline__ bool tc_finish(const TcPhase<UP>& ph, TcBars& bars, uint32_t tmem, uint32_t& acc) {
    constexpr int M = kTcTiles;
    const MoeLayerArgs& a = ph.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, units = ph.units();
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++acc) {
        const auto x = ph.at(u);
        if (!mbar_wait_warp(a.ctl, &bars.done[acc & 1], acc / 2 & 1u, a.timeout_ns)) return false;
        tc_fence_after();
        const uint32_t d = tmem + (acc & 1) * (M * 128) + (uint32_t(warp * 32) << 16);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int in = m * ph.kTile + (UP ? warp * 16 + (lane & 15) : warp * 32 + lane), row = x.row0 + in;
            if (m * ph.kTile + (UP ? 16 : 32) * warp >= ph.span) break;  // none of this warp's
            const bool use = in < ph.span && row < ph.rows;
            for (int c0 = 0; c0 < x.count; c0 += 16) {
                float v[16];
                tc_load16(v, d + m * 128 + c0);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if constexpr (UP) {
                        // lanes 0-15 hold G's rows, 16-31 U's; each half finishes every other column
                        const float other = __shfl_xor_sync(0xffffffffu, v[i], 16);
                        const bool mine = (i & 1) == (lane >> 4);
                        if (mine && use && c0 + i < x.count)
                            store_h(a, ph.l.list[x.first + c0 + i], row, lane < 16 ? silu_mul(v[i], other) : silu_mul(other, v[i]));
                    } else {
                        if (use && c0 + i < x.count)
                            a.y[size_t(ph.l.list[x.first + c0 + i]) * a.H + row] = v[i];
                    }
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tc_arrive(&bars.read[acc & 1]);
    }
    return true;
}

__global__ void __launch_bounds__(kTcThreads, 1) k_moe_tensor(const __grid_constant__ MoeLayerArgs a) {
    extern __shared__ unsigned char s_raw[];
    __shared__ TcBars bars;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
    const uint32_t smem = (smem_u32(s_raw) + 1023u) & ~1023u;  // the swizzle's period
    const LayerLists l = layer_lists(a, s_raw + a.tensor_ring + 1024);
    const int warp = threadIdx.x >> 5;
    constexpr uint32_t kColumns = 2 * kTcTiles * 128;
    if (threadIdx.x == 0) {
        s_fail = status_failed(a.ctl);
        for (int ph = 0; ph < 2; ++ph)
            for (int i = 0; i < kTcStages; ++i) {
                mbar_init(&bars.full[ph][i], kTcCopy * 32);
                mbar_init(&bars.empty[ph][i], 1);
            }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.done[i], 1);
            mbar_init(&bars.read[i], kTcEpilogue);
        }
        mbar_init(&bars.idle, 1);
        fence_barrier_init();
    }
    __syncthreads();
    if (s_fail) return;
    const int nact = sort_assignments<kTcThreads>(a, l, kTcTokens);
    if (nact < 0) return;
    if (warp == kTcEpilogue) {  // one CTA per SM: nothing competes for the columns
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(&s_tmem)), "n"(kColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    int most = 0;  // assignments of the expert that has most
    for (int q = threadIdx.x; q < nact; q += kTcThreads) most = max(most, l.act_start[q + 1] - l.act_start[q]);
    __shared__ int s_most;
    if (threadIdx.x == 0) s_most = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    atomicMax(&s_most, most);
    __syncthreads();
    most = s_most;
    const uint32_t tmem = s_tmem;
    uint32_t acc = 0;  // accumulators begun, the same count for the issuing thread and the reading warps
    auto phase = [&](const auto& ph) {
        bool ok = true;
        if (warp < kTcEpilogue) {
            ok = tc_finish(ph, bars, tmem, acc);
        } else if (warp == kTcEpilogue) {
            if (elected()) ok = tc_issue(ph, smem, bars, tmem, acc);
            __syncwarp();
        } else {
            ok = tc_copy(ph, smem, bars);
        }
        return ok;
    };
    bool ok = phase(TcPhase<true>(a, l, nact, most));
    const TcPhase<false> down(a, l, nact, most);
    if (warp > kTcEpilogue) tc_prefetch(down);
    ok = layer_barrier(a, 1, ok);
    if (ok) ok = layer_barrier(a, 2, phase(down));
    tc_fence_before();
    __syncthreads();
    if (warp == kTcEpilogue)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(kColumns));
    if (!ok) return;
    weighted_sum<kTcThreads>(a);
    __syncthreads();
    if (threadIdx.x == 0) leave_tasks(&a.st->layer_ctr, &a.st->layer_done);
}

// Bytes left for the ring of stages beside the lists: a CTA has 227 KiB, 8 of them for the static part and alignment.
static int tc_ring_bytes(const MoeLayerArgs& a) {
    const long long left = 227 * 1024 - 8 * 1024 - (long long)layer_lists_bytes(a.E, a.A);
    return left < kTcRing ? 0 : int(left / 1024 * 1024);
}

bool layer_tensor_fits(const MoeLayerArgs& a) { return tc_ring_bytes(a) > 0; }

cudaError_t launch_layer_tensor(MoeLayerArgs a, int num_sms, cudaStream_t s) {
    a.tensor_ring = tc_ring_bytes(a);
    const size_t smem = size_t(a.tensor_ring) + 1024 + layer_lists_bytes(a.E, a.A);
    cudaError_t e = cudaFuncSetAttribute(k_moe_tensor, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    // no more CTAs than there can be units of 16 rows
    const size_t units = (size_t(std::min(a.E, a.A)) + a.A / kTcTokens) * ((size_t(std::max(a.F, a.H)) + 15) / 16);
    dim3 grid(unsigned(std::max<size_t>(1, std::min<size_t>(num_sms, units)))), block(kTcThreads);
    void* args[] = {&a};
    e = cudaLaunchCooperativeKernel(reinterpret_cast<void*>(k_moe_tensor), grid, block, args, smem, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace simcomm
