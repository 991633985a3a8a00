// Penalties for repeated tokens, biases and masks on rows of scores whose V columns are on the ranks.
//
//   x > 0 ? x / repetition : x * repetition     for a token that occurs in the row's history
//   x - frequency c - presence                  for one that occurs c > 0 times behind the prompt
//   x + bias,  -inf where the mask has no bit
//
// A CTA has some columns of a row, over the ranks' shards, and counts what of the row's history and biases falls on them: a
// word of shared memory per column or, where its columns are many more than the row can name, per place of a hash table. Bit 31 for a
// token of the prompt, bit 30 for one with a bias, below them the count of the tokens behind the prompt (whole-number
// atomics: their order does not matter; the last bias of a token is the largest place). Whoever finds a word still 0 puts
// it on a list. Then the scores are copied and masked without a look at the words: scores that nothing touches keep their bits, and
// in place they are not even read. At last a thread takes a word of the list, whose score it has read before the copy, and
// writes what the rules make of it.
//
// Bound by the scores' bytes; with few rows by the latency of history, counts and scores in turn. Measured on B200, 256 rows
// of 131072 bf16 with 1024 tokens and masks, us: with a word per column, 8192 to a CTA, 53 (the words looked at while the scores are
// copied: 56, since every warp with one such column in 256 goes the long way), and of these 15 the counts and 8 the end, which
// every CTA of a row waits for alone; with a table of 2048 places, 65536 columns to a CTA, 40 (136 MB, 3.4 TB/s), of which the
// copy alone would be 23 and the masks 7. 8 rows of 131072 fp32 with 4096 tokens, biases and masks 9.3, 33 of 50257 6.9.
#include <algorithm>

#include "common.cuh"

namespace simcomm {

constexpr int kAdjustThreads = 256;
constexpr int kAdjustAhead = 4;               // 16-byte vectors of scores in flight per thread
constexpr uint32_t kInPrompt = 0x80000000u, kHasBias = 0x40000000u;
constexpr uint32_t kNoColumn = 0xffffffffu;

// Columns [v, end) of a row that lie in one shard: where they are read and written, and how they lie in vectors.
template <int DT> struct Stretch {
    static constexpr int L = Pack16<DT>::L, D = Elem<DT>::kBytes;
    const char* in;
    char* out;
    uint32_t v, end;
    uint32_t head, vecs, rest;   // scores before the first whole vector, vectors, scores outside of them
    bool in_place;
    __device__ __forceinline__ Stretch(const AdjustArgs& a, size_t row, uint32_t v_, uint32_t v1) : v(v_) {
        const uint32_t m = uint32_t(a.m), r = v / m;
        end = min(v1, uint32_t(min((size_t(r) + 1) * a.m, a.V)));
        in = static_cast<const char*>(a.logits[r]) + (row * a.ld + (v - r * m)) * D;
        out = static_cast<char*>(a.out[r]) + (row * a.ld_out + (v - r * m)) * D;
        in_place = in == out;
        const uint32_t n = end - v, phase = uint32_t(reinterpret_cast<uintptr_t>(in) & 15);
        const bool together = phase == (reinterpret_cast<uintptr_t>(out) & 15);  // 16-byte boundaries fall on the same columns
        head = together ? min(n, ((16 - phase) & 15) / D) : n;
        vecs = (n - head) / L;
        rest = n - vecs * L;
    }
    __device__ __forceinline__ uint32_t column(uint32_t i) const { return head + i * L; }
    __device__ __forceinline__ uint4 vector(uint32_t i) const { return ld_stream_v4(in + size_t(column(i)) * D); }
};

template <int DT, bool BIAS, bool HASH> __global__ void __launch_bounds__(kAdjustThreads, 4) k_adjust(const __grid_constant__ AdjustArgs a) {
    using S = Stretch<DT>;
    constexpr int L = S::L;
    // [words], with BIAS [words] places of biases, with HASH [words] columns, then the list, 16 bits each
    extern __shared__ __align__(16) uint32_t s_words[];
    __shared__ uint32_t s_listed;
    const coll_logit_rules_t& rules = a.rules;
    const bool failed = status_failed(a.ctl);
    const size_t row = blockIdx.x / a.parts;
    const uint32_t part = blockIdx.x % a.parts;
    const uint32_t v0 = a.first + part * uint32_t(a.cols), v1 = uint32_t(min(size_t(v0) + a.cols, size_t(a.last)));
    if (v0 >= v1) return;

    // the first scores are on their way while the rules are read and the history is counted
    S s(a, row, v0, v1);
    uint4 ahead[kAdjustAhead];
    auto fetch = [&](const S& from) {
        if (!from.in_place)
#pragma unroll
            for (int q = 0; q < kAdjustAhead; ++q)
                if (q * kAdjustThreads + threadIdx.x < from.vecs) ahead[q] = from.vector(q * kAdjustThreads + threadIdx.x);
    };
    fetch(s);

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
        const int b = rules.bias_start[row], e = rules.bias_start[row + 1];
        if (b < 0 || e < b || size_t(e) > rules.bias_count) bad = true;
        else {
            bias0 = b;
            biases = e - b;
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

    // whether columns [v, v + count) of the vocabulary are allowed, a bit each
    auto allowed = [&](uint32_t v, int count) {
        const uint32_t full = (1u << count) - 1u;
        if (!mask) return full;
        const uint32_t at = v & 31u;
        uint32_t w = __ldg(mask + (v >> 5)) >> at;
        if (at + count > 32) w |= __ldg(mask + (v >> 5) + 1) << (32 - at);
        return w & full;
    };
    uint32_t bits[kAdjustAhead];
    auto fetch_bits = [&](const S& from) {
#pragma unroll
        for (int q = 0; q < kAdjustAhead; ++q) {
            const uint32_t i = q * kAdjustThreads + threadIdx.x;
            if (i < from.vecs) bits[q] = allowed(from.v + from.column(i), L);
        }
    };
    fetch_bits(s);
    uint32_t* const counts = s_words;
    uint32_t* const places = counts + a.words;
    uint32_t* const keys = places + (BIAS ? a.words : 0);
    uint16_t* const list = reinterpret_cast<uint16_t*>(keys + (HASH ? a.words : 0));
    const bool any = len > 0 || biases > 0;
    if (any) {
        for (int i = threadIdx.x * 4; i < a.words; i += kAdjustThreads * 4) {
            *reinterpret_cast<uint4*>(counts + i) = make_uint4(0, 0, 0, 0);
            if constexpr (BIAS) *reinterpret_cast<uint4*>(places + i) = make_uint4(0, 0, 0, 0);
            if constexpr (HASH) *reinterpret_cast<uint4*>(keys + i) = make_uint4(kNoColumn, kNoColumn, kNoColumn, kNoColumn);
        }
        if (threadIdx.x == 0) s_listed = 0u;
    }
    // the first of the history are on their way too
    const int by4 = rules.history_len && a.hist_vec ? len / 4 : 0;
    int4 first = make_int4(-1, -1, -1, -1);
    if (int(threadIdx.x) < by4) first = __ldg(reinterpret_cast<const int4*>(seen) + threadIdx.x);
    if (__syncthreads_or(failed)) return;

    // A word of the list, its column and its score, read where it lies.
    struct Listed {
        uint32_t word, v;
        float x;
        bool ok;
    };
    auto at = [&](uint32_t v, size_t ld) { return row * ld + (v - v / uint32_t(a.m) * uint32_t(a.m)); };
    auto listed_at = [&](uint32_t i) {
        Listed e;
        e.word = list[i];
        e.v = v0 + (HASH ? keys[e.word] : e.word);
        e.x = load_elem<DT>(a.logits[e.v / uint32_t(a.m)], at(e.v, a.ld));
        e.ok = allowed(e.v, 1) != 0u;
        return e;
    };
    uint32_t listed = 0;
    Listed own{0u, 0u, 0.0f, false};
    if (any) {
        bool wrong = false;
        const uint32_t n = v1 - v0;
        // the word of a column
        auto word_of = [&](uint32_t c) {
            if constexpr (!HASH) return c;
            uint32_t w = (c * 2654435761u) >> a.hash_shift;
            while (true) {  // ends: a row names fewer columns than the table has places
                const uint32_t was = atomicCAS(&keys[w], kNoColumn, c);
                if (was == kNoColumn || was == c) return w;
                w = (w + 1) & uint32_t(a.words - 1);
            }
        };
        auto note = [&](uint32_t w, uint32_t was) {
            if (was == 0u) list[atomicAdd(&s_listed, 1u)] = uint16_t(w);
        };
        auto one = [&](int32_t id, int i) {
            const uint32_t c = uint32_t(id) - v0;
            if (c < n) {
                const uint32_t w = word_of(c);
                note(w, i < prompt ? atomicOr(&counts[w], kInPrompt) : atomicAdd(&counts[w], 1u));
            } else if (id != -1 && uint32_t(id) >= uint32_t(a.V)) {
                wrong = true;
            }
        };
        auto four = [&](const int4& id, int i) {
            one(id.x, 4 * i);
            one(id.y, 4 * i + 1);
            one(id.z, 4 * i + 2);
            one(id.w, 4 * i + 3);
        };
        if (int(threadIdx.x) < by4) four(first, threadIdx.x);
        for (int i0 = kAdjustThreads; i0 < by4; i0 += 4 * kAdjustThreads) {  // four loads in flight
            int4 id[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + q * kAdjustThreads + int(threadIdx.x);
                id[q] = i < by4 ? __ldg(reinterpret_cast<const int4*>(seen) + i) : make_int4(-1, -1, -1, -1);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) four(id[q], i0 + q * kAdjustThreads + int(threadIdx.x));
        }
        for (int i = by4 * 4 + threadIdx.x; i < len; i += kAdjustThreads) one(__ldg(seen + i), i);
        if constexpr (BIAS)
            for (int i = threadIdx.x; i < biases; i += kAdjustThreads) {
                const int32_t id = __ldg(rules.bias_token + bias0 + i);
                const uint32_t c = uint32_t(id) - v0;
                if (c < n) {
                    const uint32_t w = word_of(c);
                    note(w, atomicOr(&counts[w], kHasBias));
                    atomicMax(&places[w], uint32_t(i));
                } else if (id != -1 && uint32_t(id) >= uint32_t(a.V)) {
                    wrong = true;
                }
            }
        if (wrong) raise_status(a.ctl, COLL_ERR_INVALID_ARG);
        __syncthreads();  // words and list are complete
        listed = s_listed;
        if (threadIdx.x < listed) own = listed_at(threadIdx.x);
    }

    constexpr uint32_t kFull = (1u << L) - 1u;
    constexpr uint32_t kNone = DT == COLL_BF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
    while (true) {
        for (uint32_t k = threadIdx.x; k < s.rest; k += kAdjustThreads) {
            const uint32_t c = k < s.head ? k : k + s.vecs * L;
            using T = typename Elem<DT>::T;
            if (!allowed(s.v + c, 1)) store_elem<DT>(s.out, c, -INFINITY);
            else if (!s.in_place) reinterpret_cast<T*>(s.out)[c] = reinterpret_cast<const T*>(s.in)[c];
        }
        for (uint32_t i0 = 0; i0 < s.vecs; i0 += kAdjustAhead * kAdjustThreads) {
#pragma unroll
            for (int q = 0; q < kAdjustAhead; ++q) {
                const uint32_t i = i0 + q * kAdjustThreads + threadIdx.x;
                if (i >= s.vecs) break;
                const uint32_t ok = bits[q];
                uint4 raw = ahead[q];
                // their places are taken by what comes after the next three
                const uint32_t later = i + kAdjustAhead * kAdjustThreads;
                if (later < s.vecs) {
                    if (!s.in_place) ahead[q] = s.vector(later);
                    bits[q] = allowed(s.v + s.column(later), L);
                }
                if (s.in_place) {
                    if (ok == kFull) continue;
                    if (ok != 0u) raw = s.vector(i);
                }
                if (ok != kFull) {
                    uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                    for (int l = 0; l < 4; ++l) {
                        uint32_t keep;  // the bits of allowed scores
                        if constexpr (DT == COLL_BF16) keep = ((ok >> (2 * l)) & 1u) * 0xffffu | ((ok >> (2 * l + 1)) & 1u) * 0xffff0000u;
                        else keep = 0u - ((ok >> l) & 1u);
                        w[l] = (w[l] & keep) | (kNone & ~keep);
                    }
                    raw = make_uint4(w[0], w[1], w[2], w[3]);
                }
                st_v4(s.out + size_t(s.column(i)) * S::D, raw);
            }
        }
        if (s.end >= v1) break;
        s = S(a, row, s.end, v1);
        fetch(s);
        fetch_bits(s);
    }
    if (listed == 0) return;
    __syncthreads();  // the scores that the next ones go over are written
    for (uint32_t i = threadIdx.x; i < listed; i += kAdjustThreads) {
        const Listed e = i < kAdjustThreads ? own : listed_at(i);
        if (!e.ok) continue;  // masked, and written
        const uint32_t word = counts[e.word], count = word & ~(kInPrompt | kHasBias);
        float x = e.x;
        if (word & ~kHasBias) x = x > 0.0f ? x / repetition : x * repetition;
        if (count) x = x - frequency * float(count) - presence;
        if (BIAS && (word & kHasBias)) x += rules.bias_value[bias0 + int(places[e.word])];
        store_elem<DT>(a.out[e.v / uint32_t(a.m)], at(e.v, a.ld_out), x);
    }
}

cudaError_t launch_adjust(const AdjustArgs& args, int dtype, int num_sms, cudaStream_t s) {
    AdjustArgs a = args;
    const bool bias = a.rules.bias_start != nullptr, one = a.ranks < a.p;  // a rank view has its own shard
    a.first = one ? uint32_t(std::min(size_t(a.rank0) * a.m, a.V)) : 0u;
    a.last = one ? uint32_t(std::min((size_t(a.rank0) + 1) * a.m, a.V)) : uint32_t(a.V);
    if (a.first == a.last) return cudaSuccess;
    // Columns of a CTA: as many as leave four CTAs to an SM, 2048 at least, in whole 64s, which keeps the vectors of shards whole.
    const size_t span = a.last - a.first, wanted = std::max<size_t>(1, size_t(4 * num_sms) / a.rows);
    size_t cols = std::max<size_t>(2048, (span + wanted - 1) / wanted);
    // Columns that a row can name: a hash table with twice as many places, where that is less than a word per column; the table
    // has 8192 places at most, a CTA with a word per column 8192 columns (with biases) or 16384. What a row can name goes by the sizes of the
    // arrays, not by what it does name: 256 rows of 131072 bf16 with 1024 tokens and masks, us by the width of the history's rows: up to
    // 2048 39, 4096 61, 8192 and more 68; with 20 biases to a row (5120 in all) 94.
    const size_t names = (a.rules.history_len ? a.rules.ld_history : 0) + (bias ? a.rules.bias_count : 0);
    size_t places = 256;
    while (places < 2 * names && places < 16384) places *= 2;
    const bool hash = places <= 8192 && places * 2 < cols;
    if (!hash) cols = std::min<size_t>(cols, bias ? 8192 : 16384);
    cols = (cols + 63) / 64 * 64;
    a.cols = uint32_t(cols);
    a.words = int(hash ? places : cols);
    a.hash_shift = 32;
    for (size_t q = 1; q < places; q *= 2) --a.hash_shift;
    a.parts = uint32_t((span + cols - 1) / cols);
    const size_t ctas = a.rows * a.parts;
    if (ctas > size_t(INT32_MAX)) return cudaErrorInvalidValue;
    const size_t smem = size_t(a.words) * (4 + (bias ? 4 : 0) + (hash ? 4 : 0) + 2);
    auto go = [&](auto kernel) {
        if (smem > 47 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
            if (e != cudaSuccess) return e;
        }
        kernel<<<unsigned(ctas), kAdjustThreads, smem, s>>>(a);
        return cudaGetLastError();
    };
    auto table = [&](auto dt, auto b) {
        constexpr int DT = decltype(dt)::value;
        constexpr bool B = decltype(b)::value;
        return hash ? go(k_adjust<DT, B, true>) : go(k_adjust<DT, B, false>);
    };
    using Bf = std::integral_constant<int, COLL_BF16>;
    using Fp = std::integral_constant<int, COLL_FP32>;
    if (dtype == COLL_BF16) return bias ? table(Bf{}, std::true_type{}) : table(Bf{}, std::false_type{});
    return bias ? table(Fp{}, std::true_type{}) : table(Fp{}, std::false_type{});
}

}  // namespace simcomm
