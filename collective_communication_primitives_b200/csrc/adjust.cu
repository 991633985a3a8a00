// Penalties for repeated tokens, biases and masks on rows of scores whose V columns are on the ranks.
//
//   x > 0 ? x / repetition : x * repetition     for a token that occurs in the row's history
//   x - frequency c - presence                  for one that occurs c > 0 times behind the prompt
//   x + bias,  -inf where the mask has no bit
//
// A CTA has some columns of a row and a word of shared memory for each: bit 31 for a token of the prompt, below it the
// count of the tokens behind it. It reads the row's whole history and counts what falls on its columns (whole-number
// atomics, so their order does not matter), likewise the biases (the last entry of a token is the largest place), and
// then goes over its columns once. Scores that nothing touches keep their bits; in place they are not even read. Bound
// by the scores' bytes; with few rows by the latency of history, counts and scores in turn. The history is read once per
// CTA, from L2: a longer one is worth more columns to a CTA.
#include <algorithm>

#include "common.cuh"

namespace simcomm {

constexpr int kAdjustThreads = 256;
constexpr int kAdjustAhead = 4;               // 16-byte vectors of scores in flight per thread
constexpr uint32_t kInPrompt = 0x80000000u;

template <int DT, bool BIAS> __global__ void __launch_bounds__(kAdjustThreads) k_adjust(const __grid_constant__ AdjustArgs a) {
    using P = Pack16<DT>;
    constexpr int L = P::L, D = Elem<DT>::kBytes;
    extern __shared__ __align__(16) uint32_t s_words[];  // [cols + 4] counts, then, with BIAS, [cols + 4] places of biases
    const coll_logit_rules_t& rules = a.rules;
    const bool failed = status_failed(a.ctl);
    size_t b = blockIdx.x;
    const size_t tile = b % a.tiles;
    b /= a.tiles;
    const int r = a.rank0 + int(b % a.ranks);
    const size_t row = b / a.ranks;
    const size_t c0 = tile * a.cols, v0 = size_t(r) * a.m + c0;  // first column in the shard's row and in the vocabulary
    if (v0 >= a.V) return;
    const uint32_t n = uint32_t(min(min(size_t(a.cols), a.m - c0), a.V - v0));
    const char* in = static_cast<const char*>(a.logits[r]) + (row * a.ld + c0) * D;
    char* out = static_cast<char*>(a.out[r]) + (row * a.ld_out + c0) * D;
    const bool in_place = in == out;
    const uintptr_t phase = reinterpret_cast<uintptr_t>(in) & 15;
    const bool together = phase == (reinterpret_cast<uintptr_t>(out) & 15);  // 16-byte boundaries fall on the same columns
    const uint32_t head = together ? min(n, uint32_t((16 - phase) & 15) / D) : n;
    const uint32_t vecs = (n - head) / L, rest = n - vecs * L;

    // the first scores are on their way while the history is counted
    uint4 ahead[kAdjustAhead];
    if (!in_place)
#pragma unroll
        for (int q = 0; q < kAdjustAhead; ++q) {
            const uint32_t i = q * kAdjustThreads + threadIdx.x;
            if (i < vecs) ahead[q] = ld_stream_v4(in + (size_t(head) + size_t(i) * L) * D);
        }

    // the row's rules; one that is out of range is reported and left out
    bool bad = false;
    const int32_t* seen = nullptr;
    int len = 0, prompt = 0;
    if (rules.history_len) {
        len = rules.history_len[row];
        prompt = rules.prompt_len ? rules.prompt_len[row] : 0;
        if (len < 0 || size_t(len) > rules.ld_history || prompt < 0 || prompt > len) {
            bad = true;
            len = 0;
        }
        seen = rules.history + row * rules.ld_history;
    }
    int bias0 = 0, biases = 0;
    if constexpr (BIAS) {
        const int s = rules.bias_start[row], e = rules.bias_start[row + 1];
        if (s < 0 || e < s || size_t(e) > rules.bias_count) bad = true;
        else {
            bias0 = s;
            biases = e - s;
        }
    }
    const uint32_t* mask = nullptr;
    if (rules.mask) {
        const long long k = rules.mask_row ? (long long)rules.mask_row[row] : (long long)row;
        if (k < -1 || k >= (long long)rules.mask_rows) bad = true;
        else if (k >= 0) mask = rules.mask + size_t(k) * rules.ld_mask;
    }
    if (bad && threadIdx.x == 0) raise_status(a.ctl, COLL_ERR_INVALID_ARG);
    const float repetition = rules.repetition ? rules.repetition[row] : 1.0f;
    const float frequency = rules.frequency ? rules.frequency[row] : 0.0f;
    const float presence = rules.presence ? rules.presence[row] : 0.0f;

    // column head is at a 16-byte boundary of the words
    uint32_t* const counts = s_words + ((4 - (head & 3)) & 3);
    uint32_t* const places = counts + a.cols + 4;
    const bool any = len > 0 || biases > 0;
    if (any) {
        const int words = (int(a.cols) + 4) * (BIAS ? 2 : 1);
        for (int i = threadIdx.x * 4; i < words; i += kAdjustThreads * 4) *reinterpret_cast<uint4*>(s_words + i) = make_uint4(0, 0, 0, 0);
    }
    if (__syncthreads_or(failed)) return;
    if (any) {
        bool wrong = false;
        auto meet = [&](int32_t id, int i) {
            const uint32_t c = uint32_t(id) - uint32_t(v0);
            if (c < n) {
                if (i < prompt) atomicOr(&counts[c], kInPrompt);
                else atomicAdd(&counts[c], 1u);
            } else if (id != -1 && uint32_t(id) >= uint32_t(a.V)) {
                wrong = true;
            }
        };
        const int by4 = a.hist_vec ? len / 4 : 0;
#pragma unroll 4
        for (int i = threadIdx.x; i < by4; i += kAdjustThreads) {
            const int4 id = __ldg(reinterpret_cast<const int4*>(seen) + i);
            meet(id.x, 4 * i);
            meet(id.y, 4 * i + 1);
            meet(id.z, 4 * i + 2);
            meet(id.w, 4 * i + 3);
        }
        for (int i = by4 * 4 + threadIdx.x; i < len; i += kAdjustThreads) meet(__ldg(seen + i), i);
        if constexpr (BIAS)
            for (int i = threadIdx.x; i < biases; i += kAdjustThreads) {
                const int32_t id = __ldg(rules.bias_token + bias0 + i);
                const uint32_t c = uint32_t(id) - uint32_t(v0);
                if (c < n) atomicMax(&places[c], uint32_t(i) + 1u);
                else if (id != -1 && uint32_t(id) >= uint32_t(a.V)) wrong = true;
            }
        if (wrong) raise_status(a.ctl, COLL_ERR_INVALID_ARG);
        __syncthreads();
    }

    auto changed = [&](float x, uint32_t count, uint32_t place) {
        if (count) x = x > 0.0f ? x / repetition : x * repetition;
        count &= ~kInPrompt;
        if (count) x = x - frequency * float(count) - presence;
        if (BIAS && place) x += rules.bias_value[bias0 + int(place) - 1];
        return x;
    };
    // whether columns [c, c + count) are allowed, a bit each
    auto allowed = [&](uint32_t c, int count) {
        const uint32_t full = (1u << count) - 1u;
        if (!mask) return full;
        const uint32_t v = uint32_t(v0) + c, at = v & 31u;
        uint32_t w = __ldg(mask + (v >> 5)) >> at;
        if (at + count > 32) w |= __ldg(mask + (v >> 5) + 1) << (32 - at);
        return w & full;
    };

    for (uint32_t k = threadIdx.x; k < rest; k += kAdjustThreads) {
        const uint32_t c = k < head ? k : k + vecs * L;
        const uint32_t count = any ? counts[c] : 0u, place = BIAS && any ? places[c] : 0u;
        const bool ok = allowed(c, 1);
        if (!ok) {
            store_elem<DT>(out, c, -INFINITY);
        } else if (count | place) {
            store_elem<DT>(out, c, changed(load_elem<DT>(in, c), count, place));
        } else if (!in_place) {
            using T = typename Elem<DT>::T;
            reinterpret_cast<T*>(out)[c] = reinterpret_cast<const T*>(in)[c];
        }
    }
    constexpr uint32_t kFull = (1u << L) - 1u;
    constexpr uint32_t kNone = DT == COLL_BF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
    for (uint32_t i0 = 0; i0 < vecs; i0 += kAdjustAhead * kAdjustThreads) {
        if (i0 > 0 && !in_place)
#pragma unroll
            for (int q = 0; q < kAdjustAhead; ++q) {
                const uint32_t i = i0 + q * kAdjustThreads + threadIdx.x;
                if (i < vecs) ahead[q] = ld_stream_v4(in + (size_t(head) + size_t(i) * L) * D);
            }
#pragma unroll
        for (int q = 0; q < kAdjustAhead; ++q) {
            const uint32_t i = i0 + q * kAdjustThreads + threadIdx.x;
            if (i >= vecs) break;
            const uint32_t c = head + i * L;
            uint32_t count[L], place[L], touched = 0u;
#pragma unroll
            for (int l = 0; l < L; ++l) count[l] = place[l] = 0u;
            if (any) {
#pragma unroll
                for (int l = 0; l < L; l += 4) {
                    const uint4 w = *reinterpret_cast<const uint4*>(counts + c + l);
                    count[l] = w.x, count[l + 1] = w.y, count[l + 2] = w.z, count[l + 3] = w.w;
                    if constexpr (BIAS) {
                        const uint4 o = *reinterpret_cast<const uint4*>(places + c + l);
                        place[l] = o.x, place[l + 1] = o.y, place[l + 2] = o.z, place[l + 3] = o.w;
                    }
                }
#pragma unroll
                for (int l = 0; l < L; ++l) touched |= count[l] | place[l];
            }
            const uint32_t ok = allowed(c, L);
            if (in_place && !touched && ok == kFull) continue;
            char* const to = out + size_t(c) * D;
            if (ok == 0u) {
                st_v4(to, make_uint4(kNone, kNone, kNone, kNone));
                continue;
            }
            const uint4 raw = in_place ? ld_stream_v4(in + size_t(c) * D) : ahead[q];
            uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            if (touched) {
                float x[L];
                P::unpack(raw, x);
#pragma unroll
                for (int l = 0; l < L; ++l) {
                    if (!(count[l] | place[l])) continue;
                    const float y = changed(x[l], count[l], place[l]);
                    if constexpr (DT == COLL_BF16) {
                        const uint32_t bits = float_to_bf16_bits(y);
                        w[l / 2] = l % 2 ? (w[l / 2] & 0xffffu) | (bits << 16) : (w[l / 2] & 0xffff0000u) | bits;
                    } else {
                        w[l] = __float_as_uint(y);
                    }
                }
            }
            if (ok != kFull)
#pragma unroll
                for (int l = 0; l < L; ++l)
                    if (!((ok >> l) & 1u)) {
                        if constexpr (DT == COLL_BF16)
                            w[l / 2] = l % 2 ? (w[l / 2] & 0xffffu) | 0xff800000u : (w[l / 2] & 0xffff0000u) | 0xff80u;
                        else
                            w[l] = 0xff800000u;
                    }
            st_v4(to, make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
}

cudaError_t launch_adjust(const AdjustArgs& args, int dtype, int num_sms, cudaStream_t s) {
    AdjustArgs a = args;
    const bool bias = a.rules.bias_start != nullptr;
    // Columns of a CTA.
    const size_t most = bias ? 16384 : 32768;
    size_t cols = 8192;
    while (cols > 2048 && a.rows * a.ranks * ((a.m + cols - 1) / cols) < size_t(2 * num_sms)) cols /= 2;
    while (cols < most && cols < a.m && a.rules.history_len && a.rules.ld_history > 4 * cols) cols *= 2;
    a.cols = int(cols);
    a.tiles = int((a.m + cols - 1) / cols);
    const size_t ctas = a.rows * a.ranks * a.tiles;
    if (ctas > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    const size_t smem = (cols + 4) * 4 * (bias ? 2 : 1);
    auto go = [&](auto kernel) {
        if (smem > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
            if (e != cudaSuccess) return e;
        }
        kernel<<<unsigned(ctas), kAdjustThreads, smem, s>>>(a);
        return cudaGetLastError();
    };
    if (dtype == COLL_BF16) return bias ? go(k_adjust<COLL_BF16, true>) : go(k_adjust<COLL_BF16, false>);
    return bias ? go(k_adjust<COLL_FP32, true>) : go(k_adjust<COLL_FP32, false>);
}

}  // namespace simcomm
