// The next token of every row of logits (exq_sample) for gfx950: temperature,
// top-k, top-p and min-p from given random numbers.
//
// With M the row's largest logit and T its temperature, token i weighs
//   w_i = e^{(l_i - M) / T} = 2^t,  t = (l_i - M) log2(e) / T,
// computed in 64 bits (whose products run at the rate of 32 here) and held as a
// whole number of units of 2^-shift.  Sums of whole numbers do not depend on
// their order, so the kernel may add weights through LDS atomics and still give
// the same token every time; and 2^-45 units keep a border between two tokens
// where the real numbers have it.
//
// One workgroup takes a row.  The tokens a filter may keep are found without
// sorting: the j-th largest of the threads' own largest logits is a threshold
// that at least j logits reach and, with the row dealt out over 1024 threads, not
// many more.  These go to LDS, where the cut is found digit by digit of their
// values (a histogram of weights or counts for each digit), and the draw digit
// by digit of their indices.  Only where the cut lies below them (nearly flat
// rows, or a top-k in the thousands) is the whole row histogrammed.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "exq_device_common.h"
#include "exq_internal.h"
#include "exq_operand.h"

namespace exq {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int kSampleThreads = 1024, kSampleWaves = kSampleThreads / 64;
constexpr int kSampleList = 8192;             // candidates that LDS holds
constexpr int kSampleEach = kSampleList / kSampleThreads;
constexpr int kSampleBins = 2048;             // of a digit of 11 bits
constexpr int kSampleMaxVocabLog2 = 21;

// A setting of every row: from memory, or the same for all.
template <class T> struct PerRow {
    const T* p;
    T all;
    __device__ T of(int row) const { return p ? p[row] : all; }
};

struct SampleArgs {
    const void* logits;
    int64_t stride;   // elements
    int rows, vocab, shift;
    const float* u;
    PerRow<float> temperature;
    PerRow<int32_t> top_k;
    PerRow<float> top_p, min_p;
    int32_t* tokens;
    float* logprobs;
};

// Ordered keys: larger for larger logits, the value in the upper bits; 0 for a
// NaN or -infinity, which are never drawn.  -0 and 0 have one key.
template <class T> struct Logit;
template <> struct Logit<_Float16> {
    typedef h8 vec;
    static constexpr int VEC = 8, LEVELS = 2;   // digits of 11 bits that tell keys apart
    __device__ static uint32_t key(_Float16 x) {
        uint32_t b = __builtin_bit_cast(uint16_t, x);
        if (b == 0x8000u) b = 0;
        const uint32_t k = b ^ (b & 0x8000u ? 0xFFFFu : 0x8000u);
        return (float)x > -__builtin_huge_valf() ? k << 16 : 0u;
    }
    __device__ static float value(uint32_t key) {
        const uint32_t k = key >> 16;
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(k ^ (k & 0x8000u ? 0x8000u : 0xFFFFu)));
    }
};
template <> struct Logit<float> {
    typedef f4 vec;
    static constexpr int VEC = 4, LEVELS = 3;
    __device__ static uint32_t key(float x) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
        return x > -__builtin_huge_valf() ? b ^ (b & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u) : 0u;
    }
    __device__ static float value(uint32_t k) { return __builtin_bit_cast(float, k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu)); }
};

// Weights of a row.  2^f for |f| <= 1/2 from its series: the first term left
// out, (f ln 2)^13 / 13!, is below 2^-52.
struct Weights {
    double top, c;   // largest logit, log2(e) / T
    float topf;
    double scale;    // 2^shift
    double least;    // min-p, 0 for none
    __device__ double real(float l) const {
#pragma clang fp contract(off)   // the same bits wherever the compiler puts it
        double t = l == topf ? 0.0 : ((double)l - top) * c;
        t = __builtin_fmax(t, -1100.0);
        const double n = __builtin_rint(t), f = (t - n) * 0.69314718055994530942;
        double p = 1.0 / 479001600;
        p = __builtin_fma(p, f, 1.0 / 39916800);
        p = __builtin_fma(p, f, 1.0 / 3628800);
        p = __builtin_fma(p, f, 1.0 / 362880);
        p = __builtin_fma(p, f, 1.0 / 40320);
        p = __builtin_fma(p, f, 1.0 / 5040);
        p = __builtin_fma(p, f, 1.0 / 720);
        p = __builtin_fma(p, f, 1.0 / 120);
        p = __builtin_fma(p, f, 1.0 / 24);
        p = __builtin_fma(p, f, 1.0 / 6);
        p = __builtin_fma(p, f, 0.5);
        p = __builtin_fma(p, f, 1.0);
        p = __builtin_fma(p, f, 1.0);
        return __builtin_ldexp(p, (int)n);
    }
    // In units, rounded: 2^52 + w * 2^shift has the whole number in its lower bits.
    __device__ uint64_t units(double w) const {
        return __builtin_bit_cast(uint64_t, __builtin_fma(w, scale, 4503599627370496.0)) & 0xFFFFFFFFFFFFFull;
    }
    __device__ uint64_t of(float l) const { return units(real(l)); }
    // ln of its probability among weights of `sum` units
    __device__ float log_of(float l, float temperature, uint64_t sum) const {
        const double z = l == topf ? 0.0 : ((double)l - top) / (double)temperature;
        return (float)(z - log((double)sum / scale));
    }
    // Zero below min-p.
    __device__ uint64_t kept(float l) const {
        const double w = real(l);
        return w >= least || l == topf ? units(w) : 0;
    }
};

struct SampleShared {
    union {
        uint64_t list[kSampleList];                          // key and index of a candidate
        uint64_t tiles[(1 << kSampleMaxVocabLog2) / 256 + 2];   // sums of weights
    };
    uint64_t bins[kSampleBins];
    uint64_t wave[kSampleWaves];
    uint64_t above;
    uint32_t bin, count;
};

__device__ __forceinline__ uint64_t wave_sum_before(uint64_t x, uint64_t& total) {   // exclusive
    const int lane = threadIdx.x & 63;
    uint64_t s = x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint64_t y = __shfl_up(s, d);
        if (lane >= d) s += y;
    }
    total = __shfl(s, 63);
    return s - x;
}

// Sum over the workgroup, and of the threads before.
__device__ __forceinline__ uint64_t block_sum_before(SampleShared& s, uint64_t x, uint64_t& total) {
    const int wave = threadIdx.x / 64;
    uint64_t mine;
    uint64_t before = wave_sum_before(x, mine);
    __syncthreads();
    if (threadIdx.x % 64 == 0) s.wave[wave] = mine;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        before += w < wave ? s.wave[w] : 0;
        total += s.wave[w];
    }
    return before;
}
__device__ __forceinline__ uint64_t block_sum(SampleShared& s, uint64_t x) {
    uint64_t total;
    block_sum_before(s, x, total);
    return total;
}

// The largest key K with sum of amounts of keys >= K at least `need` (which
// all reach), from LEVELS digits of 11 bits below bit TOP, to the last one looked
// at; `above`: the sum of amounts of larger ones.  source(f) calls
// f(key, amount) for the thread's elements.
template <int TOP, int LEVELS, class S>
__device__ __forceinline__ uint32_t select_key(SampleShared& s, uint64_t need, uint64_t& above, S&& source) {
    const int t = threadIdx.x;
    uint32_t key = 0;
    above = 0;
#pragma unroll
    for (int level = 0; level < LEVELS; ++level) {
        const int low = TOP - 11 * (level + 1) > 0 ? TOP - 11 * (level + 1) : 0;   // of this digit
        const int high = TOP - 11 * level;
        __syncthreads();
        s.bins[t] = s.bins[t + kSampleThreads] = 0;
        __syncthreads();
        source([&](uint32_t k, uint64_t amount) {
            const bool match = level == 0 || ((k ^ key) >> high) == 0;
            if (match && amount)
                atomicAdd(reinterpret_cast<unsigned long long*>(&s.bins[(k >> low) & (kSampleBins - 1) & ((1u << (high - low)) - 1)]),
                          (unsigned long long)amount);
        });
        __syncthreads();
        // bins from the top, two a thread
        const int b = kSampleBins - 1 - 2 * t;
        const uint64_t x = s.bins[b], y = s.bins[b - 1];
        uint64_t total;
        const uint64_t before = above + block_sum_before(s, x + y, total);
        if (before < need && need <= before + x + y) {
            const bool first = need <= before + x;
            s.bin = first ? b : b - 1;
            s.above = first ? before : before + x;
        }
        __syncthreads();
        key |= s.bin << low;
        above = s.above;
    }
    return key;
}

template <class T> __device__ __forceinline__ int head_elements(const T* row, int vocab) {
    return min(vocab, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T));
}

// f(index, value) for the thread's elements of the row, in ascending order.
template <class T, class F> __device__ __forceinline__ void for_row(const T* row, int vocab, F&& f) {
    typedef typename Logit<T>::vec vec;
    constexpr int VEC = Logit<T>::VEC;
    const int t = threadIdx.x, head = head_elements(row, vocab), vecs = (vocab - head) / VEC, tail = head + vecs * VEC;
    if (t < head) f(t, row[t]);
    const EXQ_GLOBAL vec* body = gptr<vec>(row + head);
    for (int j = t; j < vecs; j += 4 * kSampleThreads) {
        vec x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = j + i * kSampleThreads < vecs ? body[j + i * kSampleThreads] : vec{};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j + i * kSampleThreads < vecs)
#pragma unroll
                for (int e = 0; e < VEC; ++e) f(head + (j + i * kSampleThreads) * VEC + e, x[i][e]);
    }
    if (t < vocab - tail) f(tail + t, row[tail + t]);
}

template <class T> __global__ __launch_bounds__(kSampleThreads) void sample_kernel(SampleArgs a) {
    __shared__ SampleShared s;
    typedef Logit<T> L;
    const int t = threadIdx.x, r = blockIdx.x, lane = t % 64;
    const float u = a.u[r];
    if (u < 0.0f) return;
    const T* row = static_cast<const T*>(a.logits) + (int64_t)r * a.stride;
    const float temperature = a.temperature.of(r), top_p = a.top_p.of(r), min_p = a.min_p.of(r);
    const int top_k = a.top_k.of(r);
    const auto answer = [&](int token, float logprob) {
        a.tokens[r] = token;
        if (a.logprobs) a.logprobs[r] = logprob;
    };
    if (!(temperature >= 0.0f) || u != u || top_p != top_p || min_p != min_p) {
        if (t == 0) answer(-1, __builtin_nanf(""));
        return;
    }

    // the largest logit, at its lowest index
    uint64_t best = 0;
    for_row<T>(row, a.vocab, [&](int i, T x) {
        const uint32_t k = L::key(x);
        if (k > (uint32_t)(best >> 32)) best = (uint64_t)k << 32 | (uint32_t)~i;
    });
    const uint32_t mine = (uint32_t)(best >> 32);
#pragma unroll
    for (int d = 32; d; d /= 2) best = std::max<uint64_t>(best, __shfl_xor((unsigned long long)best, d));
    if (lane == 0) s.wave[t / 64] = best;
    if (t == 0) s.count = s.bin = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) best = std::max<uint64_t>(best, s.wave[w]);
    if (best == 0) {   // nothing that may be drawn
        if (t == 0) answer(-1, __builtin_nanf(""));
        return;
    }
    if (temperature == 0.0f || top_k == 1 || top_p <= 0.0f || min_p > 1.0f) {
        if (t == 0) answer((int)~(uint32_t)best, 0.0f);
        return;
    }
    Weights w;
    w.topf = L::value((uint32_t)(best >> 32));
    w.top = w.topf;
    w.c = 1.4426950408889634074 / (double)temperature;
    w.scale = (double)(1ull << a.shift);
    w.least = min_p;

    const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.0f;
    uint32_t cut = 1;             // kept: keys above it, and of those equal the ones up to index cut_index
    uint32_t cut_index = 0xFFFFFFFFu;
    if (by_k || by_p) {
        // candidates: at least as many as threads' maxima reach the threshold
        uint64_t above;
        const uint64_t threads = block_sum(s, mine ? 1 : 0);
        const uint64_t want = std::min<uint64_t>(by_k ? (uint64_t)top_k : 1000, threads);
        const uint32_t least = std::max(1u, select_key<32, 1>(s, want, above, [&](auto&& f) {
            if (mine) f(mine, 1);
        }));
        uint64_t sum = 0;
        for_row<T>(row, a.vocab, [&](int i, T x) {
            const uint32_t k = L::key(x);
            if (!by_k && k) sum += w.of(L::value(k));
            if (k >= least) {
                const uint32_t at = atomicAdd(&s.count, 1u);
                if (at < kSampleList) s.list[at] = (uint64_t)k << 32 | (uint32_t)i;
            }
        });
        uint64_t total = by_k ? 0 : block_sum(s, sum);   // of what top-p is a share of, if it is the whole row
        __syncthreads();
        const uint32_t count = s.count;
        uint32_t keys[kSampleEach], at[kSampleEach];
        uint64_t ws[kSampleEach];
        bool held = count <= kSampleList && (!by_k || count >= (uint32_t)top_k);
        if (held) {
            uint64_t here = 0;
#pragma unroll
            for (int i = 0; i < kSampleEach; ++i) {
                const bool in = t + i * kSampleThreads < (int)count;
                const uint64_t x = in ? s.list[t + i * kSampleThreads] : 0;
                keys[i] = (uint32_t)(x >> 32);
                at[i] = (uint32_t)x;
                ws[i] = in ? w.of(L::value(keys[i])) : 0;
                here += ws[i];
            }
            const uint64_t sum_here = block_sum(s, here);
            if (!by_k) held = (double)sum_here >= (double)top_p * (double)total;
        }
        const auto each = [&](auto&& f) {
#pragma unroll
            for (int i = 0; i < kSampleEach; ++i)
                if (keys[i]) f(keys[i], at[i], ws[i]);
        };
        const auto every = [&](auto&& f) {
            for_row<T>(row, a.vocab, [&](int i, T x) {
                const uint32_t k = L::key(x);
                if (k) f(k, (uint32_t)i, k);
            });
        };
        // Narrows the cut by one filter: `from(f)` calls f(key, index, what weighs it).
        const auto narrow = [&](auto&& from, auto&& weigh, bool counts, uint64_t need) {
            const uint32_t old = cut, old_index = cut_index;
            const auto source = [&](auto&& f) {
                from([&](uint32_t k, uint32_t i, auto x) {
                    if (k > old || (k == old && i <= old_index)) f(k, i, counts ? 1 : weigh(k, x));
                });
            };
            cut = select_key<32, L::LEVELS>(s, need, above, [&](auto&& f) { source([&](uint32_t k, uint32_t, uint64_t x) { f(k, x); }); });
            // of equal ones the first: their amounts are equal
            const uint64_t one = counts ? 1 : w.of(L::value(cut));
            const uint64_t ties = (need - above + one - 1) / one;
            uint64_t skipped;
            const uint32_t last = select_key<22, 2>(s, ties, skipped, [&](auto&& f) {
                source([&](uint32_t k, uint32_t i, uint64_t) {
                    if (k == cut) f(~i & 0x3FFFFFu, 1);
                });
            });
            cut_index = ~last & 0x3FFFFFu;
        };
        const auto filters = [&](auto&& from, auto&& weigh) {
            if (by_k) {
                uint64_t n = 0;
                from([&](uint32_t, uint32_t, auto) { ++n; });
                n = block_sum(s, n);
                narrow(from, weigh, true, std::min<uint64_t>(n, top_k));
                if (by_p) {
                    uint64_t x = 0;
                    from([&](uint32_t k, uint32_t i, auto y) {
                        if (k > cut || (k == cut && i <= cut_index)) x += weigh(k, y);
                    });
                    total = block_sum(s, x);
                }
            }
            if (by_p) {
                const double share = (double)top_p * (double)total;
                narrow(from, weigh, false, std::min<uint64_t>(std::max<uint64_t>((uint64_t)__builtin_ceil(share), 1), total));
            }
        };
        if (held) {
            filters(each, [](uint32_t, uint64_t x) { return x; });
            uint64_t sum = 0;
#pragma unroll
            for (int i = 0; i < kSampleEach; ++i) {
                const bool in = keys[i] > cut || (keys[i] == cut && at[i] <= cut_index);
                ws[i] = in ? w.kept(L::value(keys[i])) : 0;
                sum += ws[i];
            }
            sum = block_sum(s, sum);
            // the draw: indices in ascending order
            const uint64_t target = std::min<uint64_t>((uint64_t)((double)u * (double)sum), sum - 1);
            const uint32_t token = ~select_key<22, 2>(s, target + 1, above, [&](auto&& f) {
                each([&](uint32_t, uint32_t i, uint64_t x) { f(~i & 0x3FFFFFu, x); });
            }) & 0x3FFFFFu;
#pragma unroll
            for (int i = 0; i < kSampleEach; ++i)
                if (keys[i] && at[i] == token)
                    answer((int)token, w.log_of(L::value(keys[i]), temperature, sum));
            return;
        }
        filters(every, [&](uint32_t k, uint32_t) { return w.of(L::value(k)); });
        __syncthreads();
    }

    // the draw over the whole row: sums of tiles, then the tile that holds it
    const auto weight = [&](T x, int i) -> uint64_t {
        const uint32_t k = L::key(x);
        return k > cut || (k == cut && (uint32_t)i <= cut_index) ? w.kept(L::value(k)) : 0;
    };
    const int head = head_elements(row, a.vocab), vecs = (a.vocab - head) / L::VEC, tail = head + vecs * L::VEC;
    const int tiles = 2 + (vecs + 63) / 64;
    // a lane's elements of a tile: VEC neighbours, or one at the row's ends
    struct Span {
        int first, n;
    };
    const auto span = [&](int tile) -> Span {
        const int j = (tile - 1) * 64 + lane;
        if (tile == 0) return {lane, lane < head};
        if (tile == tiles - 1) return {tail + lane, lane < a.vocab - tail};
        return {head + j * L::VEC, j < vecs ? L::VEC : 0};
    };
    for (int tile = t / 64; tile < tiles; tile += kSampleWaves) {
        const Span x = span(tile);
        uint64_t sum = 0, tile_sum;
        if (x.n == L::VEC) {
            const typename L::vec v = *gptr<typename L::vec>(row + x.first);
#pragma unroll
            for (int e = 0; e < L::VEC; ++e) sum += weight(v[e], x.first + e);
        } else {
            for (int e = 0; e < x.n; ++e) sum += weight(row[x.first + e], x.first + e);
        }
        wave_sum_before(sum, tile_sum);
        if (lane == 0) s.tiles[tile] = tile_sum;
    }
    __syncthreads();
    const int per = (tiles + kSampleThreads - 1) / kSampleThreads;
    uint64_t sum = 0, total;
    for (int i = t * per; i < std::min(tiles, (t + 1) * per); ++i) sum += s.tiles[i];
    uint64_t before = block_sum_before(s, sum, total);
    const uint64_t target = std::min<uint64_t>((uint64_t)((double)u * (double)total), total - 1);
    if (before <= target && target < before + sum) {
        for (int i = t * per; i < tiles; ++i) {
            if (target < before + s.tiles[i]) {
                s.bin = i;
                s.above = before;
                break;
            }
            before += s.tiles[i];
        }
    }
    __syncthreads();
    if (t >= 64) return;
    const int tile = (int)s.bin;
    const Span x = span(tile);
    uint64_t lane_sum = 0, tile_sum;
    for (int e = 0; e < x.n; ++e) lane_sum += weight(row[x.first + e], x.first + e);
    uint64_t at = s.above + wave_sum_before(lane_sum, tile_sum);
    if (at <= target && target < at + lane_sum) {
        for (int e = 0; e < x.n; ++e) {
            const int i = x.first + e;
            at += weight(row[i], i);
            if (target < at) {
                answer(i, w.log_of(L::value(L::key(row[i])), temperature, total));
                break;
            }
        }
    }
}

}  // namespace exq

// =================================================================== host

using namespace exq;

extern "C" exq_status exq_sample(const void* logits, int bits, int rows, int vocab, int64_t row_stride, const float* u,
                                 const float* temperatures, float temperature, const int32_t* top_ks, int top_k,
                                 const float* top_ps, float top_p, const float* min_ps, float min_p, int32_t* tokens,
                                 float* logprobs, void* stream) {
    if (rows < 0 || vocab < 1) return fail(EXQ_ERR_INVALID_ARG, "rows=%d vocab=%d", rows, vocab);
    if (bits != 16 && bits != 32) return fail(EXQ_ERR_UNSUPPORTED, "logits of %d bits (16 or 32)", bits);
    if (vocab > 1 << kSampleMaxVocabLog2) return fail(EXQ_ERR_UNSUPPORTED, "vocab=%d over 2^%d", vocab, kSampleMaxVocabLog2);
    if (!temperatures && !(temperature >= 0)) return fail(EXQ_ERR_INVALID_ARG, "temperature=%g", (double)temperature);
    if (!top_ps && top_p != top_p) return fail(EXQ_ERR_INVALID_ARG, "top_p is not a number");
    if (!min_ps && min_p != min_p) return fail(EXQ_ERR_INVALID_ARG, "min_p is not a number");
    if (rows == 0) return EXQ_OK;
    if (row_stride < 0 || row_stride > kMaxStride || (rows > 1 && row_stride != 0 && row_stride < vocab))
        return fail(EXQ_ERR_INVALID_ARG, "row_stride=%lld", (long long)row_stride);
    const size_t n = 4 * (size_t)rows, size = bits / 8;
    const size_t logits_bytes = size * ((size_t)(rows - 1) * (size_t)row_stride + (size_t)vocab);
    const struct {
        const char* name;
        const void *p;
        bool needed;
    } read[] = {{"u", u, true}, {"temperatures", temperatures, false}, {"top_ks", top_ks, false}, {"top_ps", top_ps, false},
                {"min_ps", min_ps, false}},
      written[] = {{"tokens", tokens, true}, {"logprobs", logprobs, false}};
    if (!logits || !aligned(logits, size)) return fail(EXQ_ERR_INVALID_ARG, "logits is NULL or misaligned");
    for (const auto& x : read)
        if ((x.needed && !x.p) || !aligned(x.p, 4)) return fail(EXQ_ERR_INVALID_ARG, "%s is NULL or misaligned", x.name);
    for (const auto& x : written) {
        if ((x.needed && !x.p) || !aligned(x.p, 4)) return fail(EXQ_ERR_INVALID_ARG, "%s is NULL or misaligned", x.name);
        if (!x.p) continue;
        if (ranges_meet(x.p, n, logits, logits_bytes)) return fail(EXQ_ERR_INVALID_ARG, "%s overlaps logits", x.name);
        for (const auto& y : read)
            if (y.p && ranges_meet(x.p, n, y.p, n)) return fail(EXQ_ERR_INVALID_ARG, "%s overlaps %s", x.name, y.name);
    }
    if (logprobs && ranges_meet(tokens, n, logprobs, n)) return fail(EXQ_ERR_INVALID_ARG, "tokens overlaps logprobs");
    int log2 = 0;
    while ((1 << log2) < vocab) ++log2;
    const SampleArgs a{logits, row_stride, rows, vocab, std::min(51, 63 - log2), u, {temperatures, temperature},
                       {top_ks, top_k}, {top_ps, top_p}, {min_ps, min_p}, tokens, logprobs};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (bits == 16) hipLaunchKernelGGL((sample_kernel<_Float16>), dim3((unsigned)rows), dim3(kSampleThreads), 0, s, a);
    else hipLaunchKernelGGL((sample_kernel<float>), dim3((unsigned)rows), dim3(kSampleThreads), 0, s, a);
    return launched("sample launch");
}
