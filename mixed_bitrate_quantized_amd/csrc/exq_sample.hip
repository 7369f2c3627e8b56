// The next token of every row of logits (exq_sample) for gfx950: temperature,
// top-k, top-p and min-p from given random numbers.
//
// With M the row's largest logit and T its temperature, token i weighs
//   w_i = e^{(l_i - M) / T} = 2^t,  t = (l_i - M) log2(e) / T,
// computed in 64 bits and held as a whole number of units of 2^-shift.  Sums of
// whole numbers do not depend on their order, so weights may be added through LDS
// atomics and still give the same token every time; and 2^-42 to 2^-51 a unit keep a
// border between two tokens where the real numbers have it.  Where a weight counts
// for every logit of one fp16 key, sums are taken in 64-bit floating point, in a fixed
// order.
//
// One workgroup takes a row; nothing is sorted.  Every filter leaves the tokens
// above a cut: a key (a logit's bits, in order) and how many of those with that key.
//   top-k   up to 900: the k-th largest of the threads' own largest logits is a
//           threshold that at least k logits reach and, with the row dealt out over
//           1024 threads, not many more.
//   fp16    top-p, or more of top-k: a counter in LDS for every key.  The counters say
//           where top-k ends, and with a weight for every key instead of every token
//           (64-bit arithmetic takes 8 cycles an instruction: weights of 131072 tokens
//           take 36 us) what the weights add up to and where top-p ends.
//   fp32    these: a histogram of the logits, or of the weights, 64 bins for a power of
//           two.  What may be left goes to LDS, where the cut is found digit by digit
//           of the keys.
// The draw runs over what is left: up to 256 candidates are compared with one another;
// longer lists, or the row where that is too much, go through sums of tiles, then the
// tile that holds the draw.
// Rows that have to be weighed whole (no top-k; top-p or nothing) are shared out over
// several workgroups where there are few rows.
//
// The bytes of the logits are the floor (256 x 131072 fp16: 67 MB, 9.6 us).  What a call
// takes is a chain of looks with barriers between: 1 x 32000 with a top-k of 40 11.8 us,
// 16 x 50001 fp32 with settings of all kinds 26.5 (launch of the shares 9, the rest 17),
// 256 x 131072 with top-p 38: the first look 24000 cycles and 8000 until its last
// wave, the counters 13000, the end of top-p 4500, the second look, for the list,
// 28500, cut and draw 16000.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "exq_device_common.h"
#include "exq_internal.h"
#include "exq_operand.h"
#include "exq_powers.h"

namespace exq {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int kSampleThreads = 1024, kSampleWaves = kSampleThreads / 64;
constexpr int kSampleList = 4096;             // candidates that LDS holds
// A top-k that is looked for from the threads' largest logits (of 1024 threads).  So, and
// by what follows larger ones, at a top-k of 300, 600 and 890 (us):
//   1 x 32000 fp16     16.0, 18.0   17.2, 18.7   19.7, 19.2      fp32   17.0, 26.7   17.9, 28.0   20.5, 28.9
//   256 x 131072 fp16  32.9, 35.5   34.7, 36.5   38.6, 37.3      fp32   55, 91       58, 93       62, 95
constexpr int kSampleNear = 900;
// Candidates that are compared one by one, n * n / 1024 comparisons a thread.  So, and
// through the tiles of the row, 1 x 32000 fp16 by top-k alone, and with a top-p of 0.95:
//   100   11.7, 15.4   12.6, 18.5      200   13.6, 15.6   14.6, 19.0      400   22.7, 16.2   23.6, 19.5
constexpr int kSampleFew = 256;
constexpr int kDigit = 9;                     // bits looked at together
constexpr int kSampleBins = 2048;             // of a row's histogram
constexpr int kSampleParts = 16;              // of a row, at most
constexpr int kSampleCountedShare = 32768;    // logits of a part of an fp16 row with top-p, at most
// Candidates of a part; more, or more than a list together, and the row is weighed
// again.  16 x 50001 with top-p at a temperature of 32, of 256: fp16 68 us, fp32 76; of
// 512, 1024 and 2048: 32 and 34.
constexpr int kSamplePartList = 1024;
constexpr int kSampleMaxVocabLog2 = 21;
constexpr int kCounters = 1 << 15;            // of 16 bits for each sign

// A setting of every row: from memory, or the same for all.
template <class T> struct PerRow {
    const T* p;
    T all;
    __device__ __forceinline__ T of(int row) const { return p ? p[row] : all; }
};

// Words that workgroups of one launch leave for one another go past the caches of
// their XCDs.  (A fence of all waves, which writes back and drops those, took 100 us
// in 256 workgroups.)
__device__ __forceinline__ void leave(uint64_t* p, uint64_t x) { __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint64_t left_at(const uint64_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Rows shared out over `parts` workgroups each: what these leave for one another, 64
// bits each.
struct SampleSplit {
    uint64_t* p;
    int rows, parts;
    __host__ __device__ int64_t head() const { return ((int64_t)rows * (2 + parts) + 1) & ~1; }
    __device__ uint64_t* best(int r) const { return p + r; }                  // largest key, and where
    __device__ uint64_t* done(int r) const { return p + rows + r; }           // parts that are
    __device__ uint64_t* counts(int r) const { return p + 2 * rows + (int64_t)r * parts; }   // of the parts' lists
    __device__ uint64_t* bins(int r, int part) const { return p + head() + ((int64_t)r * parts + part) * kSampleBins; }
    __device__ uint64_t* tiles(int r) const { return p + head() + ((int64_t)rows * parts + r) * kSampleBins; }
    __device__ uint64_t* list(int r, int part) const {
        return p + head() + (int64_t)rows * (parts + 1) * kSampleBins + ((int64_t)r * parts + part) * kSamplePartList;
    }
    size_t bytes() const { return 8 * (size_t)(head() + (int64_t)rows * ((parts + 1) * kSampleBins + parts * kSamplePartList)); }
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
    SampleSplit split;
};

// Ordered keys: larger for larger logits; 0 for a NaN or -infinity, which are
// never drawn.  -0 and 0 have one key.
template <class T> struct Logit;
template <> struct Logit<_Float16> {
    typedef h8 vec;
    static constexpr int VEC = 8, BITS = 16, COARSE = 4;   // COARSE: bits of a key below 1/64 of a power of two
    static constexpr bool COUNTED = true;                  // a counter for every key fits LDS
    __device__ __forceinline__ static uint32_t key(_Float16 x) {
        uint32_t b = __builtin_bit_cast(uint16_t, x);
        if (b == 0x8000u) b = 0;
        const uint32_t k = b ^ (b & 0x8000u ? 0xFFFFu : 0x8000u);
        return (float)x > -__builtin_huge_valf() ? k : 0u;
    }
    __device__ __forceinline__ static float largest(const h8& x) {   // NaN aside
        const h4 a = __builtin_elementwise_max(__builtin_shufflevector(x, x, 0, 1, 2, 3), __builtin_shufflevector(x, x, 4, 5, 6, 7));
        const h2 b = __builtin_elementwise_max(__builtin_shufflevector(a, a, 0, 1), __builtin_shufflevector(a, a, 2, 3));
        return (float)__builtin_elementwise_max(b[0], b[1]);
    }
    __device__ __forceinline__ static _Float16 at(const h8& x, int e) {
        const u4v y = __builtin_bit_cast(u4v, x);
        const uint32_t pair = e < 4 ? (e < 2 ? y[0] : y[1]) : (e < 6 ? y[2] : y[3]);
        return __builtin_bit_cast(_Float16, (uint16_t)(pair >> (16 * (e & 1))));
    }
    // Key of the smallest value that is x or more (0: any).
    __device__ __forceinline__ static uint32_t first_from(double x) {
        if (!(x > -65504.0)) return 0;
        if (x > 65504.0) return 0xFC00u;
        const _Float16 near = (_Float16)(float)x;
        return key(near) + ((double)near < x);
    }
    __device__ __forceinline__ static float value(uint32_t k) {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(k ^ (k & 0x8000u ? 0x8000u : 0xFFFFu)));
    }
};
template <> struct Logit<float> {
    typedef f4 vec;
    static constexpr int VEC = 4, BITS = 32, COARSE = 17;
    static constexpr bool COUNTED = false;
    __device__ __forceinline__ static uint32_t key(float x) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
        return x > -__builtin_huge_valf() ? b ^ (b & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u) : 0u;
    }
    __device__ __forceinline__ static float largest(const f4& x) {
        return __builtin_fmaxf(__builtin_fmaxf(x[0], x[1]), __builtin_fmaxf(x[2], x[3]));
    }
    __device__ __forceinline__ static float at(const f4& x, int e) { return e < 2 ? (e ? x[1] : x[0]) : (e < 3 ? x[2] : x[3]); }
    __device__ __forceinline__ static uint32_t first_from(double x) {
        if (!(x > -(double)__FLT_MAX__)) return 0;
        if (x > (double)__FLT_MAX__) return 0xFF800000u;
        const float near = (float)x;
        return key(near) + ((double)near < x);
    }
    __device__ __forceinline__ static float value(uint32_t k) { return __builtin_bit_cast(float, k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu)); }
};

constexpr double kInfinite = 0x1p128;   // in an infinite logit's place

// Weights of a row.  A power is good to 2^-45.2, and the exponent's roundings cost a
// weight w 2^-51 |ln w|: 2^-45.9 at 2^-51.  Where up to three powers are multiplied
// (sum_counters) that makes 2^-43.3.
struct Weights {
    float topf;
    double top, c;   // largest logit (kInfinite), 256 log2(e) / T; beside an infinity all else weighs nothing
    double scale;    // 2^shift
    const double* powers;
    __device__ __forceinline__ double power(double t) const { return power_of(powers, t); }   // 2^(t / 256)
    __device__ __forceinline__ double real(float l) const {   // l: at most the largest
#pragma clang fp contract(off)
        return power((__builtin_fmin((double)l, kInfinite) - top) * c);
    }
    // In units, rounded: 2^52 + w * 2^shift has the whole number in its lower bits.
    __device__ __forceinline__ uint64_t units(double w) const {
        return __builtin_bit_cast(uint64_t, __builtin_fma(w, scale, 4503599627370496.0)) & 0xFFFFFFFFFFFFFull;
    }
    __device__ __forceinline__ uint64_t of(float l) const { return units(real(l)); }
    // ln of its probability among weights of `sum` units
    __device__ __forceinline__ float log_of(float l, float temperature, uint64_t sum) const {
        const double z = l == topf ? 0.0 : ((double)l - top) / (double)temperature;
        return (float)(z - log((double)sum / scale));
    }
};

constexpr int kSampleTiles = 2048;   // of a row, at most
static_assert(kSampleTiles == kSampleBins, "either fills a part's sums");

struct SampleShared {
    union {
        uint32_t counts[kCounters];      // of magnitude m: positive in the lower half, negative in the upper
        struct {
            uint64_t list[kSampleList], weights[kSampleList];   // of candidates: key and index, weight
            uint32_t vectors[kSampleList];                      // of the row, that hold candidates
            uint64_t tile_sum[kSampleTiles];                    // weights left, above the cut
            uint32_t tile_equal[kSampleTiles];                  // elements at it
        };
    };
    uint64_t bins[kSampleBins];
    double powers[kPowers];
    uint64_t wave[kSampleWaves];
    uint64_t below;
    uint32_t bin, count, vector_count;
    // counters' sums: for each power of two (and sign), the largest values first
    double block_weight[64];
    uint32_t block_count[64];
    double tops[2][128];
    double steps[32][4];   // weights 0, 1, 2, 3 magnitudes behind one, to its own, for each power of two
    double part_count[4], part_weight[4];
    // a cut found among them
    uint32_t cut_key, cut_above, cut_equal;
    double cut_weight_above, cut_weight, cut_need;
    double log_min_p;
    // of few candidates: their places among the others, weights before them
    uint32_t rank[kSampleFew];
    uint64_t before[kSampleFew];
};

// Over the workgroup: the sum of the threads before (with BEFORE), and of all.
template <class Op = Sum, bool BEFORE = false>
__device__ __forceinline__ uint64_t reduce(SampleShared& s, uint64_t x, uint64_t* before = nullptr) {
    static_assert(kSampleWaves == 16, "a row of lanes adds up the waves");
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const uint64_t sums = prefix64<Op>(x);
    __syncthreads();
    if (lane == 63) s.wave[wave] = sums;
    __syncthreads();
    const uint64_t waves = prefix16<Op>(s.wave[lane & 15]);
    if (BEFORE) *before = sums - x + (wave ? lane_value(waves, wave - 1) : 0);
    return lane_value(waves, 15);
}

// The bin of 64 PER that takes the running sum from the first one to `need`
// or more, and the sum below it; by one wave, for all after a barrier.
template <int PER, class F> __device__ __forceinline__ void find_bin(SampleShared& s, uint64_t need, F&& bin_at) {
    __syncthreads();
    if (threadIdx.x < 64) {
        uint64_t x[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            x[i] = s.bins[bin_at(threadIdx.x, i)];
            sum += x[i];
        }
        uint64_t before = prefix64(sum) - sum;
        if (before < need && need <= before + sum) {
            int bin = 0;
#pragma unroll
            for (int i = 0; i < PER - 1; ++i) {
                const bool past = need > before + x[i];
                if (!past) break;
                before += x[i];
                bin = i + 1;
            }
            s.bin = PER * threadIdx.x + bin;
            s.below = before;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void add_to_bin(SampleShared& s, uint32_t bin, uint64_t amount) {
    atomicAdd(reinterpret_cast<unsigned long long*>(&s.bins[bin]), (unsigned long long)amount);
}

// The same of a row's histogram, two bins to a thread, with need(sum of all).
template <class F> __device__ __forceinline__ uint64_t find_row_bin(SampleShared& s, uint64_t x0, uint64_t x1, F&& need_of) {
    static_assert(kSampleBins == 2 * kSampleThreads, "two bins to a thread");
    uint64_t before;
    const uint64_t all = reduce<Sum, true>(s, x0 + x1, &before), need = need_of(all);
    if (before < need && need <= before + x0 + x1) {
        const bool second = need > before + x0;
        s.bin = 2 * threadIdx.x + second;
        s.below = before + (second ? x0 : 0);
    }
    __syncthreads();
    return need;
}

// The smallest D below 2^bits with a sum of amounts of d <= D of `need` or more
// (which all d reach), digit by digit; `below`: the sum of the smaller ones.
// source(f) calls f(d, amount) for the thread's elements.
template <class S>
__device__ __forceinline__ uint32_t select(SampleShared& s, int bits, uint64_t need, uint64_t& below, S&& source) {
    static_assert(kDigit == 9 && kSampleThreads >= 2 << kDigit, "two sets of bins, cleared by a thread each");
    uint32_t value = 0, set = 0;   // the other set is cleared under a digit's search
    below = 0;
    __syncthreads();
    s.bins[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll 1
    for (int high = bits, low; high > 0; high = low) {
        low = max(high - kDigit, 0);
        const bool first = high == bits;
        source([&](uint32_t d, uint64_t amount) {
            const uint32_t digit = d >> low, bin = digit & ((1u << (high - low)) - 1);
            // a lane's 8 neighbours lie 64 apart: no bank conflicts
            if ((first || (digit ^ (value >> low)) >> (high - low) == 0) && amount) add_to_bin(s, set + ((bin & 7) << 6 | bin >> 3), amount);
        });
        find_bin<8>(s, need - below, [&](int lane, int i) { return (int)set + 64 * i + lane; });
        value |= s.bin << low;
        below += s.below;
        if (threadIdx.x < 1 << kDigit) s.bins[set + threadIdx.x] = 0;
        set ^= 1 << kDigit;
    }
    return value;
}

template <class T> __device__ __forceinline__ int head_elements(const T* row, int vocab) {
    return min(vocab, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T));
}

// each(vector, index, in) for the thread's vectors of the row, AHEAD in flight (in:
// whether it has one, all lanes of a wave together), and one(value, index) for the
// ends of the row, fewer than a vector each.  Later looks at a row go BACK, from what
// the last one left in the L2.
template <class T, int AHEAD, bool BACK, class F, class G>
__device__ __forceinline__ void for_vectors(const T* row, int vocab, F&& each, G&& one) {
    typedef typename Logit<T>::vec vec;
    constexpr int VEC = Logit<T>::VEC;
    const int t = threadIdx.x, head = head_elements(row, vocab), vecs = (vocab - head) / VEC, tail = head + vecs * VEC;
    const EXQ_GLOBAL vec* body = gptr<vec>(row + head);
    const int rounds = (vecs + kSampleThreads - 1) / kSampleThreads;
    const auto place = [&](int round) { return t + (BACK ? rounds - 1 - round : round) * kSampleThreads; };
    const auto load = [&](int round) { return round < rounds && place(round) < vecs ? body[place(round)] : vec{}; };
    if constexpr (AHEAD > 4) {   // a small body: unrolled
        for (int round = 0; round < rounds; round += AHEAD) {
            vec x[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) x[i] = load(round + i);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (round + i < rounds) each(x[i], head + place(round + i) * VEC, place(round + i) < vecs);
        }
    } else {   // a large one: there once
        vec x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) x[i] = load(i);
#pragma unroll 1
        for (int round = 0; round < rounds; ++round) {
            const vec now = x[0];
#pragma unroll
            for (int i = 0; i + 1 < AHEAD; ++i) x[i] = x[i + 1];
            x[AHEAD - 1] = load(round + AHEAD);
            each(now, head + place(round) * VEC, place(round) < vecs);
        }
    }
    const int ends = head + vocab - tail;
    if (t < ends) {
        const int i = t < head ? t : tail + t - head;
        one(row[i], i);
    }
}

// f(value, index) for a vector's elements, the body there once or twice.
template <class F> __device__ __forceinline__ void for_elements(const f4& x, int i, F&& f) {
    f4 y = x;
#pragma unroll 1
    for (int e = 0; e < 4; ++e) {
        f(y[0], i + e);
        y = __builtin_shufflevector(y, y, 1, 2, 3, 0);
    }
}
template <class F> __device__ __forceinline__ void for_elements(const h8& x, int i, F&& f) {
    u4v y = __builtin_bit_cast(u4v, x);
#pragma unroll 1
    for (int e = 0; e < 8; e += 2) {
        const uint32_t pair = y[0];
        const h2 z = as_h2(pair);
        f(z[0], i + e);
        f(z[1], i + e + 1);
        y = __builtin_shufflevector(y, y, 1, 2, 3, 0);
    }
}

// f(value, index) for the thread's elements of the row.
template <class T, int AHEAD, bool BACK, class F> __device__ __forceinline__ void for_row(const T* row, int vocab, F&& f) {
    for_vectors<T, AHEAD, BACK>(row, vocab, [&](const typename Logit<T>::vec& x, int i, bool in) {
        if (in) for_elements(x, i, f);
    }, [&](T x, int i) { f(x, i); });
}

// What the filters left: keys above `key`, and of those with it the first `quota`.
struct Cut {
    uint32_t key, quota;
};
// And keys from `least` on.  (The key below 0's would be -0's, which has none.)
template <class T> __device__ __forceinline__ Cut with_least(Cut cut, uint32_t least) {
    constexpr uint32_t zero = 1u << (Logit<T>::BITS - 1);
    return least > cut.key ? Cut{least - 1 - (least == zero), 0} : cut;
}

// ------------------------------------------------------- counters of fp16 keys

__device__ __forceinline__ void clear_counters(SampleShared& s) {
    u4v* zero = reinterpret_cast<u4v*>(s.counts);
#pragma unroll
    for (int i = 0; i < kCounters / 4; i += kSampleThreads) zero[threadIdx.x + i] = u4v{0, 0, 0, 0};
    __syncthreads();
}
__device__ __forceinline__ void count(SampleShared& s, uint32_t bits) {   // of the lower half
    atomicAdd(&s.counts[bits & 0x7FFFu], bits & 0x8000u ? 0x10000u : 1u);
}

// Four neighbouring magnitudes of one sign, from the largest logit to the smallest.
struct Four {
    uint32_t n[4], key[4], all;
    double w[4];
};

// From the counters `c` of magnitudes m0 .. m0 + 3.
template <bool NEGATIVE> __device__ __forceinline__ Four four_from(const u4v& c, uint32_t m0) {
    Four x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int at = NEGATIVE ? e : 3 - e;
        const uint32_t m = m0 + at;
        x.n[e] = NEGATIVE ? c[at] >> 16 : c[at] & 0xFFFFu;
        if (m == 0) x.n[e] = NEGATIVE ? 0 : x.n[e] + (c[at] >> 16);   // -0 counts as 0
        if (NEGATIVE ? m >= 0x7C00u : m > 0x7C00u) x.n[e] = 0;        // -infinity, NaN
        x.key[e] = NEGATIVE ? 0x7FFFu - m : 0x8000u | m;
    }
    x.all = x.n[0] + x.n[1] + x.n[2] + x.n[3];
    return x;
}

// The lane's of 256 magnitudes, part `part` of 4 of power of two `block`, the
// largest logits in the first lanes.
__device__ __forceinline__ Four four_of(const SampleShared& s, bool negative, int block, int part) {
    const int lane = threadIdx.x & 63, m0 = 1024 * block + 256 * (negative ? part : 3 - part) + 4 * (negative ? lane : 63 - lane);
    const u4v c = *reinterpret_cast<const u4v*>(&s.counts[m0]);
    return negative ? four_from<true>(c, m0) : four_from<false>(c, m0);
}

// Their weights, and what the counted ones add up to.  Neighbours' weights have
// one ratio within a power of two.
__device__ __forceinline__ double weigh(const SampleShared& s, const Weights& w, uint32_t top_key, int block, Four& x) {
    x.w[0] = x.w[1] = x.w[2] = x.w[3] = 0;
    if (x.all == 0) return 0.0;
    // (the first ones may lie above the largest logit, uncounted)
    const uint32_t first = std::min(x.key[0], top_key);
    const int skip = (int)(x.key[0] - first);
    const double base = w.real(Logit<_Float16>::value(first));
    double sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x.w[e] = x.n[e] ? base * s.steps[block][max(e - skip, 0)] : 0.0;
        sum = __builtin_fma((double)x.n[e], x.w[e], sum);
    }
    return sum;
}

// Adds the counters up by power of two and sign, their weights too if asked for.
// The number of logits that may be drawn; -1: a counter overflowed (65536 equal ones).
__device__ __forceinline__ int sum_counters(SampleShared& s, const Weights& w, uint32_t top_key, bool weights, int vocab) {
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t / 64), lane = t & 63;
    if (weights && t < 32 * 4)   // neighbours of a power of two lie 2^(block - 25) apart
        s.steps[t / 4][t % 4] = w.power(-(t % 4) * __builtin_ldexp(w.c, max(t / 4, 1) - 25));
    // the weight of the largest value of 256 magnitudes (whatever it is above the largest logit)
    if (weights && t < 256) s.tops[t / 128][t % 128] = w.real(Logit<_Float16>::value(t < 128 ? 0x80FFu + 256 * t : 0x7FFFu - 256 * (t - 128)));
    __syncthreads();
    uint64_t all = 0;
#pragma unroll 1
    for (int block = wave; block < 32; block += kSampleWaves) {
        uint32_t n[2] = {0, 0};
        double sum[2] = {0, 0};
        // of four magnitudes 4 i behind the largest of 256
        const double behind = weights ? w.power(-4.0 * lane * __builtin_ldexp(w.c, max(block, 1) - 25)) : 0.0, ahead = __shfl(behind, 63 - lane);
        const double s1 = s.steps[block][1], s2 = s.steps[block][2], s3 = s.steps[block][3];
#pragma unroll 1
        for (int quarter = 4 * block; quarter < 4 * block + 4; ++quarter) {
            const uint32_t m0 = 256 * quarter + 4 * lane;
            const u4v c = *reinterpret_cast<const u4v*>(&s.counts[m0]);
            if (__ballot((c[0] | c[1] | c[2] | c[3]) != 0) == 0) continue;
            // 0, infinities and NaN, or values above the largest logit among them
            if (quarter == 0 || block == 31 || quarter == (int)((top_key & 0x8000u ? top_key & 0x7FFFu : 0x7FFFu - top_key) >> 8)) {
                Four x = four_from<false>(c, m0);
                n[0] += x.all;
                if (weights) sum[0] += weigh(s, w, top_key, block, x);
                x = four_from<true>(c, m0);
                n[1] += x.all;
                if (weights) sum[1] += weigh(s, w, top_key, block, x);
                continue;
            }
            uint32_t low[4], high[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                low[e] = c[e] & 0xFFFFu;
                high[e] = c[e] >> 16;
            }
            const uint32_t lows = low[0] + low[1] + low[2] + low[3], highs = high[0] + high[1] + high[2] + high[3];
            n[0] += lows;
            n[1] += highs;
            if (!weights) continue;
            if (__ballot(lows != 0)) {
                const double x = __builtin_fma(s1, (double)low[2], (double)low[3]), y = __builtin_fma(s3, (double)low[0], s2 * (double)low[1]);
                sum[0] = __builtin_fma(s.tops[0][quarter] * ahead, x + y, sum[0]);
            }
            if (__ballot(highs != 0)) {
                const double x = __builtin_fma(s1, (double)high[1], (double)high[0]), y = __builtin_fma(s3, (double)high[3], s2 * (double)high[2]);
                sum[1] = __builtin_fma(s.tops[1][quarter] * behind, x + y, sum[1]);
            }
        }
        const uint64_t both = prefix64((uint64_t)n[1] << 32 | n[0]);
        all += n[0] + n[1];
        const double up = weights ? prefix64(sum[0]) : 0.0, down = weights ? prefix64(sum[1]) : 0.0;
        if (lane == 63) {
            s.block_count[31 - block] = (uint32_t)both;
            s.block_count[32 + block] = (uint32_t)(both >> 32);
            s.block_weight[31 - block] = up;
            s.block_weight[32 + block] = down;
        }
    }
    // -infinity and NaN were not counted above
    uint64_t rest = 0;
    for (int m = 0x7C00 + t; m < kCounters; m += kSampleThreads) rest += (s.counts[m] >> 16) + (m > 0x7C00 ? s.counts[m] & 0xFFFFu : 0);
    const uint64_t both = reduce(s, all | rest << 32);
    return (both & 0xFFFFFFFFu) + (both >> 32) == (uint64_t)vocab ? (int)(uint32_t)both : -1;
}

// Where the running sum of counts, or weights, reaches `need` (with `share`: that
// share of all weights): into s.cut_*.  Four waves take a part each of the power of
// two that holds it.
__device__ __forceinline__ void find_key(SampleShared& s, const Weights& w, uint32_t top_key, bool counts, double need, bool weights,
                                         bool share) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const auto at_lane = [](double x, int i) { return __builtin_bit_cast(double, lane_value(__builtin_bit_cast(uint64_t, x), i)); };
    double n_before = 0, w_before = 0, here = 0, here_w = 0, here_to = 0, here_w_to = 0;
    Four x{};
    __syncthreads();
    if (wave < 4) {
        const double n = s.block_count[lane], weight = s.block_weight[lane];
        const double n_to = prefix64(n), w_to = prefix64(weight);
        if (share) need *= at_lane(w_to, 63);
        // (the last block that holds anything, if rounding kept the sum below)
        const uint64_t reach = __ballot((counts ? n_to : w_to) >= need && n > 0), any = __ballot(n > 0);
        const int at = reach ? __builtin_ctzll(reach) : 63 - __builtin_clzll(any);
        n_before = at_lane(n_to - n, at);
        w_before = at_lane(w_to - weight, at);
        const int block = at >= 32 ? at - 32 : 31 - at;
        x = four_of(s, at >= 32, block, wave);
        here = x.all;
        here_w = weights ? weigh(s, w, top_key, block, x) : 0.0;
        here_to = prefix64(here);
        here_w_to = prefix64(here_w);
        if (lane == 63) {
            s.part_count[wave] = here_to;
            s.part_weight[wave] = here_w_to;
        }
    }
    __syncthreads();
    if (wave < 4) {
        double n = n_before, weight = w_before;
#pragma unroll
        for (int part = 0; part < 4; ++part) {
            if (part == wave) {
                n_before = n;
                w_before = weight;
            }
            n += s.part_count[part];
            weight += s.part_weight[part];
        }
        if (wave == 0 && lane == 0) s.cut_need = need;
        need = __builtin_fmin(need, counts ? n : weight);
        const double from = counts ? n_before : w_before, own = counts ? here_to : here_w_to;
        // the first part, and its first lane, that reach it and hold something
        const uint64_t found = __ballot(x.all != 0 && from + own >= need);
        if (from < need && found && lane == __builtin_ctzll(found)) {
            double nb = n_before + (here_to - here), wb = w_before + (here_w_to - here_w);
            bool done = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!x.n[e] || done) continue;
                s.cut_key = x.key[e];
                s.cut_above = (uint32_t)nb;
                s.cut_equal = x.n[e];
                s.cut_weight_above = wb;
                s.cut_weight = weights ? x.w[e] : 0.0;
                nb += x.n[e];
                if (weights) wb += x.n[e] * x.w[e];
                done = (counts ? nb : wb) >= need;
            }
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- candidates

__device__ __forceinline__ uint64_t share_of(float top_p, uint64_t total) {   // what top-p needs of it
    return std::min<uint64_t>(std::max<uint64_t>((uint64_t)__builtin_ceil((double)top_p * (double)total), 1), total);
}
__device__ __forceinline__ uint64_t target_of(float u, uint64_t total) {
    return std::min<uint64_t>((uint64_t)((double)__builtin_fminf(u, 1.0f) * (double)total), total - 1);
}

// What is known of a row, and what is left to do on its list of candidates.
struct Row {
    int count;           // of candidates
    int vocab;
    uint32_t top_key;
    int key_bits;        // candidates' keys lie within 2^key_bits of the top
    int top_k;           // 0: done
    float top_p;         // 1 or more: done
    Cut cut;
    uint32_t least;      // the smallest key that min-p leaves
    float u, temperature;
};

// Up to kSampleFew candidates: every one is compared with every other, by all
// threads, which gives each its place in the filters' order and in the index's.
// Weights put there leave a sum over the threads before for either.
template <class T, class A>
__device__ __forceinline__ void finish_few(SampleShared& s, const Weights& w, const Row& f, A&& answer) {
    typedef Logit<T> L;
    const int t = threadIdx.x, n = f.count <= 64 ? 64 : f.count <= 128 ? 128 : kSampleFew;
    const int i = t & (n - 1), group = t / n, per = n * n / kSampleThreads;
    const bool one = t < f.count;   // the thread has the list's t-th
    const uint64_t x = i < f.count ? s.list[i] : 0;
    const uint32_t key = (uint32_t)(x >> 32), index = (uint32_t)x;
    const uint64_t weight = one ? w.of(L::value(key)) : 0;
    if (t < n) s.rank[t] = 0;
    __syncthreads();
    const int first_j = group * per, last_j = std::min(f.count, first_j + per);
    uint32_t rank = 0;
#pragma unroll 4
    for (int j = first_j; j < last_j; ++j) {
        const uint64_t y = s.list[j];
        rank += ((y ^ 0xFFFFFFFFu) > (x ^ 0xFFFFFFFFu) ? 1u : 0u) + ((uint32_t)y < index ? 0x10000u : 0u);
    }
    if (rank && i < f.count) atomicAdd(&s.rank[i], rank);
    __syncthreads();
    const uint32_t place = one ? s.rank[t] & 0xFFFFu : 0, at = one ? s.rank[t] >> 16 : 0;
    uint32_t limit = f.top_k ? std::min(f.top_k, f.count) : f.count;   // places left
    if (f.cut.key) limit = (uint32_t)std::min<uint64_t>(limit, reduce(s, one && key > f.cut.key) + f.cut.quota);
    bool in = one && place < limit;
    if (f.top_p < 1.0f) {
        if (one) s.before[place] = in ? weight : 0;
        __syncthreads();
        const uint64_t here = one ? s.before[t] : 0;
        uint64_t before;
        const uint64_t need = share_of(f.top_p, reduce<Sum, true>(s, here, &before));
        if (one) s.before[t] = before;
        __syncthreads();
        in = in && s.before[place] < need;
    }
    if (one) {
        s.list[at] = x;
        s.weights[at] = in && key >= f.least ? weight : 0;
    }
    __syncthreads();
    const uint64_t mine = one ? s.weights[t] : 0;
    uint64_t lower;
    const uint64_t sum = reduce<Sum, true>(s, mine, &lower), target = target_of(f.u, sum);
    if (mine && lower <= target && target < lower + mine) {
        const uint64_t y = s.list[t];
        answer((int)(uint32_t)y, w.log_of(L::value((uint32_t)(y >> 32)), f.temperature, sum));
    }
}

// The cut of a longer list, from the filters that are left to do.
template <class T> __device__ __forceinline__ void filter_list(SampleShared& s, const Weights& w, Row& f) {
    typedef Logit<T> L;
    // a thread's own candidates, which no other looks at
    const auto each = [&](auto&& g) {
#pragma unroll 1
        for (int i = threadIdx.x; i < f.count; i += kSampleThreads) g((uint32_t)(s.list[i] >> 32), s.weights[i]);
    };
    each([&](uint32_t k, uint64_t& x) { x = w.of(L::value(k)); });
    uint64_t below;
#pragma unroll 1
    for (int filter = f.top_k ? 0 : 1; filter < (f.top_p < 1.0f ? 2 : 1); ++filter) {
        const bool counts = filter == 0;
        uint64_t all = 0;
        each([&](uint32_t k, uint64_t x) { all += k < f.cut.key ? 0 : counts ? 1 : k > f.cut.key ? x : 0; });
        all = reduce(s, all);
        if (!counts && f.cut.key) all += f.cut.quota * w.of(L::value(f.cut.key));
        const uint64_t need = counts ? (uint64_t)f.top_k : share_of(f.top_p, all);
        if (need >= all) continue;
        const uint32_t key = f.top_key - select(s, f.key_bits, need, below, [&](auto&& g) {
            each([&](uint32_t k, uint64_t x) {
                if (k >= f.cut.key) g(f.top_key - k, counts ? 1 : x);
            });
        });
        const uint64_t one = counts ? 1 : w.of(L::value(key));
        f.cut = Cut{key, (uint32_t)((need - below + one - 1) / one)};
    }
    if (f.cut.key == 0) {   // the whole list is left, and the draw looks at the row: from the list's smallest key on
        uint64_t rest = 0;
        each([&](uint32_t k, uint64_t) { rest = std::max<uint64_t>(rest, ~k); });
        f.cut = Cut{~(uint32_t)reduce<Larger>(s, rest), 0xFFFFFFFFu};
    }
}

// The row in tiles: its head, groups of 64 vectors (a wave's look), its tail.
template <class T> struct Tiles {
    int head, vecs, tail, vocab, groups, per, count;   // per: groups of a tile
    __device__ __forceinline__ Tiles(const T* row, int n) {
        constexpr int VEC = Logit<T>::VEC;
        vocab = n;
        head = head_elements(row, n);
        vecs = (n - head) / VEC;
        tail = head + vecs * VEC;
        groups = (vecs + 63) / 64;
        per = groups <= kSampleTiles - 2 ? 1 : (groups + kSampleTiles - 3) / (kSampleTiles - 2);
        count = 2 + (groups + per - 1) / per;
    }
    __device__ __forceinline__ int of(int i) const {   // of index i
        if (i < head) return 0;
        const int group = (i - head) / (64 * Logit<T>::VEC);
        return i >= tail ? count - 1 : 1 + (per == 1 ? group : group / per);
    }
};

// -------------------------------------------------------------------- kernel

// The tiles of a row's body that a part of it has, and each(value, index) for their
// elements and, for the first part, the row's ends; put(tile) behind a wave's
// elements of a tile.
template <class T> struct Part {
    int first, last;   // tiles of the body, from 0
    __device__ __forceinline__ Part(const Tiles<T>& tiles, int part, int parts) {
        const int body = tiles.count - 2, each = (body + parts - 1) / parts;
        first = std::min(body, part * each);
        last = std::min(body, first + each);
    }
    template <class F, class G>
    __device__ __forceinline__ void each(const Tiles<T>& tiles, const T* row, int part, F&& f, G&& put) const {
        typedef typename Logit<T>::vec vec;
        constexpr int VEC = Logit<T>::VEC;
        const int t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
        const EXQ_GLOBAL vec* body = gptr<vec>(row + tiles.head);
        const int end = std::min(last * tiles.per, tiles.groups);
        // the next group's load is under way while one is worked on
        const auto load = [&](int group) { return group < end && group * 64 + lane < tiles.vecs ? body[group * 64 + lane] : vec{}; };
        int group = first * tiles.per + wave;
        vec next = load(group);
#pragma unroll 1
        for (; group < end; group += kSampleWaves) {
            const vec x = next;
            next = load(group + kSampleWaves);
            const int j = group * 64 + lane;
            if (j < tiles.vecs) for_elements(x, tiles.head + j * VEC, f);
            put(1 + (tiles.per == 1 ? group : group / tiles.per));
        }
        if (part == 0 && t < 64) {
            if (t < tiles.head) f(row[t], t);
            put(0);
            if (t < tiles.vocab - tiles.tail) f(row[tiles.tail + t], tiles.tail + t);
            put(tiles.count - 1);
        }
    }
    // s.tile_sum of them, and of the row's ends
    __device__ __forceinline__ void clear(SampleShared& s, const Tiles<T>& tiles) const {
        for (int i = 1 + first + threadIdx.x; i < 1 + last; i += kSampleThreads) s.tile_sum[i] = 0;
        if (threadIdx.x < 2) s.tile_sum[threadIdx.x ? tiles.count - 1 : 0] = 0;
    }
    __device__ __forceinline__ void store(const SampleShared& s, const Tiles<T>& tiles, int part, uint64_t* out) const {
        for (int i = 1 + first + threadIdx.x; i < 1 + last; i += kSampleThreads) leave(out + i, s.tile_sum[i]);
        if (part == 0 && threadIdx.x < 2) {
            const int i = threadIdx.x ? tiles.count - 1 : 0;
            leave(out + i, s.tile_sum[i]);
        }
    }
};
// A wave's sum, to its tile.
__device__ __forceinline__ void put_sum(SampleShared& s, uint64_t& sum, int tile) {
    if (__ballot(sum != 0)) {
        sum = prefix64(sum);
        if (threadIdx.x % 64 == 63) atomicAdd(reinterpret_cast<unsigned long long*>(&s.tile_sum[tile]), (unsigned long long)sum);
    }
    sum = 0;
}

// A part's share of the first look: the weights of its tiles, by tile, or with
// BINS by bin_of(logit).
template <class T, bool BINS, class B>
__device__ __forceinline__ void sum_part(SampleShared& s, const SampleSplit& split, const T* row, int vocab, int r, int part,
                                         const Weights& w, B&& bin_of) {
    const Tiles<T> tiles(row, vocab);
    const Part<T> mine(tiles, part, split.parts);
    __syncthreads();
    if (BINS) s.bins[threadIdx.x] = s.bins[threadIdx.x + kSampleThreads] = 0;
    else mine.clear(s, tiles);
    __syncthreads();
    uint64_t sum = 0;
    mine.each(tiles, row, part, [&](T x, int) {
        if ((float)x > -__builtin_huge_valf()) {
            const uint64_t amount = w.of((float)x);
            if (!BINS) sum += amount;
            else if (amount) add_to_bin(s, (uint32_t)bin_of((float)x), amount);
        }
    }, [&](int tile) {
        if (!BINS) put_sum(s, sum, tile);
    });
    __syncthreads();
    if (BINS) {
        uint64_t* out = split.bins(r, part);
        for (int i = threadIdx.x; i < kSampleBins; i += kSampleThreads) *gptr_w<uint64_t>(out + i) = s.bins[i];
    } else {
        mine.store(s, tiles, part, split.tiles(r));
    }
}

// A part's share of the second: the weights of its tiles' logits of smaller bins than
// `bin`, where top-p ends, that min-p leaves (from `least`), and a list of those
// of that bin.  Whether all other parts were done before, with theirs.
template <class T, class B>
__device__ __forceinline__ bool cut_part(SampleShared& s, const SampleSplit& split, const T* row, int vocab, int r, int part,
                                         const Weights& w, B&& bin_of, int bin, uint32_t least) {
    typedef Logit<T> L;
    const int t = threadIdx.x;
    const Tiles<T> tiles(row, vocab);
    const Part<T> mine(tiles, part, split.parts);
    mine.clear(s, tiles);
    if (t == 0) s.count = 0;
    __syncthreads();
    uint64_t sum = 0;
    mine.each(tiles, row, part, [&](T x, int i) {
        if (!((float)x > -__builtin_huge_valf())) return;
        const int b = bin_of((float)x);
        if (b > bin) return;
        if (b < bin) {
            if (L::key(x) >= least) sum += w.of((float)x);
        } else {
            const uint32_t at = atomicAdd(&s.count, 1u);
            if (at < kSamplePartList) s.list[at] = (uint64_t)L::key(x) << 32 | (uint32_t)i;
        }
    }, [&](int tile) { put_sum(s, sum, tile); });
    __syncthreads();
    mine.store(s, tiles, part, split.tiles(r));
    const int n = (int)s.count;
    uint64_t* out = split.list(r, part);
    for (int i = t; i < std::min(n, kSamplePartList); i += kSampleThreads) leave(out + i, s.list[i]);
    if (t == 0) leave(split.counts(r) + part, (uint64_t)n);
    // The last one goes on.  What a part leaves has arrived before its one in `done`, and
    // is read behind the last one's.
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (t == 0) s.count = (uint32_t)__hip_atomic_fetch_add(split.done(r), 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    return (int)s.count == split.parts - 1;
}

// The parts' lists as one; whether they are whole and fit it.
__device__ __forceinline__ bool join_lists(SampleShared& s, const SampleSplit& split, int r, int& count) {
    const int lane = threadIdx.x & 63;
    const uint64_t n = lane < split.parts ? left_at(split.counts(r) + lane) : 0;
    const uint64_t upto = prefix64(n);
    if (__ballot(n > kSamplePartList) || lane_value(upto, 63) > kSampleList) return false;
    count = (int)lane_value(upto, 63);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    static_assert(kSampleParts <= kSampleWaves, "a wave to a part");
    if (wave < split.parts) {
        const int from = (int)(lane_value(upto, wave) - lane_value(n, wave)), own = (int)lane_value(n, wave);
        const uint64_t* x = split.list(r, wave);
        for (int i = lane; i < own; i += 64) s.list[from + i] = left_at(x + i);
    }
    __syncthreads();
    return true;
}

// A workgroup to a row.  Rows whose every logit has to be weighed are shared out over
// split.parts of them if there are.  A launch before (FIRST) has all of them look for
// the largest logit and each weigh a part.  Then one of them draws, or, with top-p,
// each does that part's logits at and above the end of it and the last one draws.
// Rows that are not split have their one workgroup beside these.
template <class T, bool FIRST> __global__ __launch_bounds__(kSampleThreads) void sample_kernel(SampleArgs a) {
    __shared__ SampleShared s;
    typedef Logit<T> L;
    typedef typename L::vec vec;
    const int t = threadIdx.x, lane = t % 64, part = blockIdx.x / a.rows, r = blockIdx.x - part * a.rows;
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
        if (!FIRST && part == 0 && t == 0) answer(-1, __builtin_nanf(""));
        return;
    }
    const bool first_only = temperature == 0.0f || top_k == 1 || top_p <= 0.0f || min_p > 1.0f;
    const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.0f;
    const bool near = by_k && top_k <= kSampleNear;   // top-k from the threads' largest logits
    // (fp16's counters cost less than weighing a large part of a row twice)
    const bool split = a.split.parts > 1 && !(L::COUNTED && by_p && a.vocab > kSampleCountedShare * a.split.parts) && !first_only && !by_k && (by_p || !(min_p > 0.0f));
    if (split ? !FIRST && !by_p && part : FIRST || part) return;   // what one workgroup has all of
    bool counted = L::COUNTED && !split && !first_only && !near && (by_k || by_p);
    if (t < kPowers) s.powers[t] = exp2_series((double)t / kPowers);
    if (t == 0) s.bin = s.below = 0;
    if (t == kPowers && min_p > 0.0f) s.log_min_p = log((double)min_p);
    if (counted) clear_counters(s);

    float mine = -__builtin_huge_valf();   // the thread's largest logit, in which vector it comes first
    int mine_at = 0;
    uint32_t mine_key = 0;
    uint64_t best;
    if (!FIRST && split) {
        best = *a.split.best(r);
        __syncthreads();
    } else {
        for_vectors<T, 6, false>(row, a.vocab, [&](const vec& x, int i, bool in) {
            if (!in) return;
            const float most = L::largest(x);
            if (most > mine) {
                mine = most;
                mine_at = i;
            }
            if constexpr (L::COUNTED) {
                if (counted) {
                    const u4v bits = __builtin_bit_cast(u4v, x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        count(s, bits[e]);
                        count(s, bits[e] >> 16);
                    }
                }
            }
        }, [&](T x, int i) {
            // the row's first elements come behind its vectors: of equal logits the lower index
            if ((float)x > mine || ((float)x == mine && i < mine_at)) {
                mine = (float)x;
                mine_at = i;
            }
            if constexpr (L::COUNTED) {
                if (counted) count(s, __builtin_bit_cast(uint16_t, x));
            }
        });
        mine_key = L::key((T)mine);
        best = reduce<Larger>(s, mine_key ? (uint64_t)mine_key << 32 | (uint32_t)~mine_at : 0);
    }
    if (FIRST && part == 0 && t == 0) {
        *a.split.best(r) = best;
        *a.split.done(r) = 0;
    }
    if (best == 0) {   // nothing that may be drawn
        if (!FIRST && part == 0 && t == 0) answer(-1, __builtin_nanf(""));
        return;
    }
    const uint32_t top_key = (uint32_t)(best >> 32);
    if (first_only) {
        const int i = (int)~(uint32_t)best + t;
        if (t < 64) {
            const uint64_t is = __ballot(t < L::VEC && i < a.vocab && L::key(row[min(i, a.vocab - 1)]) == top_key);
            if (t == 0) answer(i + __builtin_ctzll(is), 0.0f);
        }
        return;
    }
    const float topf = L::value(top_key), finite_top = __builtin_fminf(topf, __FLT_MAX__);
    const Weights w{topf, __builtin_fmin((double)topf, kInfinite), topf > __FLT_MAX__ ? 1e300 : kPowers * 1.4426950408889634074 / (double)temperature,
                    (double)(1ull << a.shift), s.powers};
    Row f{0, a.vocab, top_key, L::BITS, 0, 1.0f, Cut{0, 0xFFFFFFFFu}, 0, u, temperature};
    if (min_p > 0.0f) {   // w >= min-p where the logit is M + T ln(min-p) or more
        // (at an infinite temperature all weigh 1: infinity times ln(min-p), 0 for 1, is no number from which on)
        const double least = min_p == 1.0f && temperature <= __FLT_MAX__ ? (double)topf : (double)topf + (double)temperature * s.log_min_p;
        f.least = L::first_from(least);
    }

    // 64 bins for one of the logits, or for a power of two of the weights
    const auto bins_of = [&](bool counts) {
        const float rate = counts ? 64.0f : __builtin_fminf((float)(w.c * (64.0 / kPowers)), 1e30f);
        return [=](float l) {
            const float d = (finite_top - __builtin_fminf(l, __FLT_MAX__)) * rate;
            return d < (float)(kSampleBins - 1) ? (int)d : kSampleBins - 1;
        };
    };
    if constexpr (FIRST) {
        if (by_p) sum_part<T, true>(s, a.split, row, a.vocab, r, part, w, bins_of(false));
        else sum_part<T, false>(s, a.split, row, a.vocab, r, part, w, bins_of(false));
        return;
    }

    // Elements that want(value) asks for, which no NaN or -infinity passes, into the
    // list: first the vectors that hold one (any(vector) tells, or may), then their elements.
    const auto collect = [&](auto&& any, auto&& want) __attribute__((always_inline)) {
        __syncthreads();
        if (t == 0) s.count = s.vector_count = 0;
        __syncthreads();
        // places for all of a wave's at once
        const auto places = [&](uint32_t* counter) {
            const uint64_t all = __ballot(true);
            const uint32_t before = __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
            uint32_t at = 0;
            if (before == 0) at = atomicAdd(counter, (uint32_t)__builtin_popcountll(all));
            return __builtin_amdgcn_readfirstlane(at) + before;
        };
        const auto put = [&](T x, int i) {
            const uint32_t at = places(&s.count);
            if (at < kSampleList) s.list[at] = (uint64_t)L::key(x) << 32 | (uint32_t)i;
        };
        for_vectors<T, 6, true>(row, a.vocab, [&](const vec& x, int i, bool in) {
            if (in && any(x)) {
                const uint32_t at = places(&s.vector_count);
                if (at < kSampleList) s.vectors[at] = (uint32_t)i;
            }
        }, [&](T x, int i) {
            if (want(x)) put(x, i);
        });
        __syncthreads();
        const int n = (int)std::min<uint32_t>(s.vector_count, 0x7FFFFFFFu);
        if (n > kSampleList) return n;
#pragma unroll 1
        for (int j = t; j < n; j += kSampleThreads) {
            const int i = (int)s.vectors[j];
            const vec x = *gptr<vec>(row + i);
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < L::VEC; ++e) hits |= want(x[e]) ? 1u << e : 0;
            while (hits) {
                const int e = __builtin_ctz(hits);
                put(L::at(x, e), i + e);
                hits &= hits - 1;
            }
        }
        __syncthreads();
        return (int)std::min<uint32_t>(s.count, 0x7FFFFFFFu);
    };
    const T nothing = (T)-__builtin_huge_valf();
    const auto collect_from = [&](uint32_t key) __attribute__((always_inline)) {   // 0: all
        const T from = key ? (T)L::value(key) : nothing;
        return collect([&](const vec& x) { return key ? L::largest(x) >= (float)from : L::largest(x) > (float)from; },
                       [&](T x) { return key ? x >= from : x > from; });
    };

    uint64_t bins[2] = {0, 0};   // of the row's histogram, the thread's two
    bool summed = split && !by_p;   // whether the parts' sums of tiles hold what is left
    if (split && by_p) {
        typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
#pragma unroll 8
        for (int p = 0; p < a.split.parts; ++p) {
            const u64x2 x = *gptr<u64x2>(a.split.bins(r, p) + 2 * t);
            bins[0] += x[0];
            bins[1] += x[1];
        }
        const uint64_t need = find_row_bin(s, bins[0], bins[1], [&](uint64_t all) { return share_of(top_p, all); });
        const int bin = (int)s.bin;
        const uint64_t behind = need - s.below;
        if (!cut_part<T>(s, a.split, row, a.vocab, r, part, w, bins_of(false), bin, f.least)) return;
        summed = join_lists(s, a.split, r, f.count);
        if (summed) {
            // the bin's keys lie close together
            uint32_t most = 0, rest = 0;
            for (int i = t; i < f.count; i += kSampleThreads) {
                const uint32_t k = (uint32_t)(s.list[i] >> 32);
                most = std::max(most, k);
                rest = std::max(rest, ~k);
            }
            most = (uint32_t)reduce<Larger>(s, most);
            rest = most - ~(uint32_t)reduce<Larger>(s, rest);
            uint64_t skipped;
            const uint32_t key = most - select(s, rest ? 32 - __builtin_clz(rest) : 0, behind, skipped, [&](auto&& g) {
                for (int i = t; i < f.count; i += kSampleThreads) {
                    const uint32_t k = (uint32_t)(s.list[i] >> 32);
                    g(most - k, w.of(L::value(k)));
                }
            });
            const uint64_t one = w.of(L::value(key));
            f.cut = Cut{key, (uint32_t)((behind - skipped + one - 1) / one)};
        }
    }
    bool held = false;   // whether the list holds all that the filters can leave
    if (!summed && (by_k || by_p || f.least)) {
        if (!by_k && !by_p) {
            f.count = collect_from(f.least);
            held = f.count <= kSampleList;
        }
        if (near) {
            // a threshold that top_k threads' largest logits reach, to 1/64 of a power of two
            const auto coarse = [&](uint32_t k) { return min((top_key >> L::COARSE) - (k >> L::COARSE), (1u << kDigit) - 1); };
            const uint64_t want = std::min<uint64_t>(top_k, reduce(s, mine_key ? 1 : 0));
            uint64_t below;
            const uint32_t least = select(s, kDigit, want, below, [&](auto&& g) {
                if (mine_key) g(coarse(mine_key), 1);
            });
            const bool any = least == (1u << kDigit) - 1;
            f.count = collect_from(any ? 0 : ((top_key >> L::COARSE) - least) << L::COARSE);
            held = f.count <= kSampleList && (any || f.count >= top_k);
            f.top_k = top_k;
            f.top_p = top_p;
            if (!any) f.key_bits = L::COARSE + kDigit;
        }
        if constexpr (L::COUNTED) {
            // With top-k, top-p is left to the list if that can hold what top-k leaves.
            bool weights = by_p && !(by_k && top_k <= kSampleList / 2);
            uint32_t kept = 0;   // at the cut or above
#pragma unroll 1
            while (counted) {
                const int some = sum_counters(s, w, top_key, weights, a.vocab);
                counted = some >= 0;
                if (!counted) break;
                kept = (uint32_t)some;
                if (by_k && some > top_k) {
                    find_key(s, w, top_key, true, (double)top_k, weights, false);
                    f.cut = Cut{s.cut_key, (uint32_t)top_k - s.cut_above};
                    kept = s.cut_above + s.cut_equal;
                }
                if (weights || !by_p || kept <= kSampleList) break;
                weights = true;
            }
            if (counted) {
                if (weights) {
                    const bool cut = f.cut.key != 0;
                    find_key(s, w, top_key, false, (double)top_p * (cut ? s.cut_weight_above + f.cut.quota * s.cut_weight : 1.0), true, !cut);
                    const double ties = __builtin_ceil((s.cut_need - s.cut_weight_above) / s.cut_weight);
                    uint32_t quota = ties < 1.0 ? 1u : ties > (double)s.cut_equal ? s.cut_equal : (uint32_t)ties;
                    if (f.cut.key == s.cut_key) quota = std::min(quota, f.cut.quota);
                    f.cut = Cut{s.cut_key, quota};
                    kept = s.cut_above + s.cut_equal;
                }
                if (kept <= kSampleList) {
                    // (what top-p is a share of includes what min-p drops)
                    const bool later = by_p && !weights;
                    f.count = collect_from(later ? f.cut.key : std::max(f.cut.key, f.least));
                    if (later) f.top_p = top_p;
                    held = true;
                }
            }
        }
        if (!counted && !held && (by_k || by_p)) {
            f.top_k = 0;
            f.top_p = 1.0f;
            f.key_bits = L::BITS;
#pragma unroll 1
            for (int filter = by_k ? 0 : 1; filter < (by_p ? 2 : 1); ++filter) {
                const bool counts = filter == 0;
                const auto bin_of = bins_of(counts);
                const bool none = f.cut.key == 0;
                const T cut = none ? nothing : (T)L::value(f.cut.key);
                const auto left = [&](T x) { return none ? x > cut : x >= cut; };
                if (!split) {
                    __syncthreads();
                    s.bins[t] = s.bins[t + kSampleThreads] = 0;
                    __syncthreads();
                    for_row<T, 4, true>(row, a.vocab, [&](T x, int) {
                        if (x > cut) {
                            const uint64_t amount = counts ? 1 : w.of((float)x);
                            if (amount) add_to_bin(s, (uint32_t)bin_of((float)x), amount);
                        }
                    });
                    if (!counts && !none && t == 0) add_to_bin(s, (uint32_t)bin_of((float)cut), f.cut.quota * w.of((float)cut));
                    __syncthreads();
                    bins[0] = s.bins[2 * t];
                    bins[1] = s.bins[2 * t + 1];
                }
                uint64_t all = 0;
                const uint64_t need = find_row_bin(s, bins[0], bins[1], [&](uint64_t sum) {
                    all = sum;
                    return counts ? (uint64_t)top_k : share_of(top_p, sum);
                });
                if (need >= all) continue;
                const int bin = (int)s.bin;
                const uint64_t before = s.below;
                // all that is left, if it fits the list; else the bin that holds the cut
                int count = 0, from = 0;
#pragma unroll 1
                for (; from <= bin; from = from < bin ? bin : bin + 1) {
                    const auto in = [&](T x) { return left(x) && bin_of((float)x) >= from && bin_of((float)x) <= bin; };
                    count = collect([&](const vec& x) {
                        bool some = false;
#pragma unroll
                        for (int e = 0; e < L::VEC; ++e) some = some || in(x[e]);
                        return some;
                    }, in);
                    if (count <= kSampleList) break;
                }
                uint64_t skipped;
                uint32_t d;
                if (count <= kSampleList) {
                    if (from == 0) {   // all that is left
                        held = true;
                        f.count = count;
                    }
                    if (held && counts) {   // top-k is left to the list, and top-p of that
                        f.top_k = top_k;
                        f.top_p = top_p;
                        break;
                    }
                    const uint64_t behind = from ? before : 0;
                    d = select(s, L::BITS, need - behind, skipped, [&](auto&& g) {
#pragma unroll 1
                        for (int i = t; i < count; i += kSampleThreads) {
                            const uint32_t k = (uint32_t)(s.list[i] >> 32);
                            g(top_key - k, counts ? 1 : w.of(L::value(k)));
                        }
                    });
                    skipped += behind;
                } else {   // equal or nearly equal ones: over the row again
                    d = select(s, L::BITS, need, skipped, [&](auto&& g) {
                        for_row<T, 4, true>(row, a.vocab, [&](T x, int) {
                            if (left(x)) g(top_key - L::key(x), counts ? 1 : w.of((float)x));
                        });
                    });
                }
                const uint64_t one = counts ? 1 : w.of(L::value(top_key - d));
                f.cut = Cut{top_key - d, (uint32_t)((need - skipped + one - 1) / one)};
            }
        }
        if (held && f.count <= kSampleFew) {
            finish_few<T>(s, w, f, answer);
            return;
        }
        if (held) filter_list<T>(s, w, f);
        __syncthreads();
    }

    // the draw: weights left, tile by tile of the row, then the tile that holds it
    const Tiles<T> tiles(row, a.vocab);
    f.cut = with_least<T>(f.cut, f.least);
    const T cut = f.cut.key ? (T)L::value(f.cut.key) : nothing;
    const uint64_t one = f.cut.key ? w.of((float)cut) : 0;   // of each of those at the cut
    for (int i = t; i < tiles.count; i += kSampleThreads) {
        s.tile_sum[i] = summed ? left_at(a.split.tiles(r) + i) : 0;
        s.tile_equal[i] = 0;
    }
    __syncthreads();
    if (summed || held) {
#pragma unroll 1
        for (int i = t; i < f.count; i += kSampleThreads) {
            const uint32_t k = (uint32_t)(s.list[i] >> 32);
            const int tile = tiles.of((int)(uint32_t)s.list[i]);
            if (k > f.cut.key) atomicAdd(reinterpret_cast<unsigned long long*>(&s.tile_sum[tile]), (unsigned long long)w.of(L::value(k)));
            else if (k == f.cut.key) atomicAdd(&s.tile_equal[tile], 1u);
        }
    } else {
        uint64_t sum = 0;
        uint32_t equal = 0;
        const auto add = [&](T l, int) {
            equal += l == cut;   // (without a cut: -infinities, of which none counts)
            if (l > cut) sum += w.of((float)l);
        };
        const auto put = [&](int tile) {
            if (__ballot(sum != 0)) {
                sum = prefix64(sum);
                if (lane == 63) atomicAdd(reinterpret_cast<unsigned long long*>(&s.tile_sum[tile]), (unsigned long long)sum);
            }
            if (__ballot(equal != 0)) {
                equal = (uint32_t)prefix64((uint64_t)equal);
                if (lane == 63) atomicAdd(&s.tile_equal[tile], equal);
            }
            sum = equal = 0;
        };
        for_vectors<T, 4, true>(row, a.vocab, [&](const vec& x, int i, bool in) {
            // (cut or not, what is below it adds nothing)
            if (__ballot(in && L::largest(x) >= (float)cut) == 0) return;
            if (in) for_elements(x, i, add);
            put(tiles.of(__builtin_amdgcn_readfirstlane(i)));
        }, [](T, int) {});
        if (t < 64) {   // the row's ends
            if (t < tiles.head) add(row[t], t);
            put(0);
            if (t < a.vocab - tiles.tail) add(row[tiles.tail + t], tiles.tail + t);
            put(tiles.count - 1);
        }
    }
    __syncthreads();
    if (t >= 64) return;

    // one wave: neighbouring tiles to a lane
    const int per = (tiles.count + 63) / 64, begin = std::min(tiles.count, lane * per), end = std::min(tiles.count, begin + per);
    const auto taken = [&](uint64_t from, uint64_t n) {   // of n at the cut behind `from` others
        return from >= f.cut.quota ? 0 : std::min<uint64_t>(n, f.cut.quota - from);
    };
    uint64_t equal = 0, sum = 0;
    for (int i = begin; i < end; ++i) equal += s.tile_equal[i];
    equal = prefix64(equal) - equal;
    const uint64_t equal_first = equal;
    for (int i = begin; i < end; ++i) {
        sum += s.tile_sum[i] + taken(equal, s.tile_equal[i]) * one;
        equal += s.tile_equal[i];
    }
    uint64_t upto = prefix64(sum);
    const uint64_t total = lane_value(upto, 63), target = target_of(u, total);
    const uint64_t reach = __ballot(target < upto);
    int tile = begin;
    uint64_t before = upto - sum;
    equal = equal_first;
    for (; tile < end - 1; ++tile) {
        const uint64_t here = s.tile_sum[tile] + taken(equal, s.tile_equal[tile]) * one;
        if (target < before + here) break;
        before += here;
        equal += s.tile_equal[tile];
    }
    const int owner = reach ? __builtin_ctzll(reach) : 63;
    tile = __builtin_amdgcn_readlane(tile, owner);
    before = lane_value(before, owner);
    equal = lane_value(equal, owner);
    // the tile's elements, 64 vectors at a time: a lane has neighbours, or one at the row's ends
    const int groups = tile == 0 || tile == tiles.count - 1 ? 1 : tiles.per;
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
        int first, n;
        if (tile == 0) {
            first = lane;
            n = lane < tiles.head;
        } else if (tile == tiles.count - 1) {
            first = tiles.tail + lane;
            n = first < a.vocab;
        } else {
            const int j = ((tile - 1) * tiles.per + g) * 64 + lane;
            first = tiles.head + j * L::VEC;
            n = j < tiles.vecs ? L::VEC : 0;
        }
        vec x{};
        if (n == L::VEC) x = *gptr<vec>(row + first);
        else if (n) x[0] = row[first];
        uint32_t lane_equal = 0;
#pragma unroll
        for (int e = 0; e < L::VEC; ++e) lane_equal += e < n && x[e] == cut;
        const uint32_t equal_to = (uint32_t)prefix64((uint64_t)lane_equal);
        uint64_t seen = equal + equal_to - lane_equal, to[L::VEC], lane_sum = 0;   // the weights up to each of the lane's
#pragma unroll
        for (int e = 0; e < L::VEC; ++e) {
            if (e < n && x[e] > cut) lane_sum += w.of((float)x[e]);
            else if (e < n && x[e] == cut) lane_sum += seen++ < f.cut.quota ? one : 0;
            to[e] = lane_sum;
        }
        const uint64_t sums = prefix64(lane_sum), from = before + sums - lane_sum;
        if (from <= target && target < from + lane_sum) {
            int e = 0;
            float l = (float)x[0];
#pragma unroll
            for (int i = 1; i < L::VEC; ++i)
                if (target >= from + to[i - 1]) {
                    e = i;
                    l = (float)x[i];
                }
            answer(first + e, w.log_of(l, temperature, total));
        }
        before += lane_value(sums, 63);
        equal += (uint32_t)__builtin_amdgcn_readlane((int)equal_to, 63);
    }
}

}  // namespace exq

// =================================================================== host

using namespace exq;

namespace {

constexpr int kSampleWorkgroups = 256;   // of a call whose rows are split: one to a CU
constexpr int kSampleSplit = 16384;      // smallest vocabulary that is
constexpr int kSampleShare = 4096;       // logits of a part, at least

// The second launch and what parts leave for one another cost 6 us.  Without and with
// it (us; drawn from all, and from a nucleus of 0.9):
//   1 x 8192 fp32    9.1, 10.6   19.5, 22.6       1 x 131072 fp16   47, 16.5   39, 30
//   1 x 16384 fp32   12.5, 11.2  25.1, 22.0       128 x 50001 fp16  23.8, 19.2   34.6, 36.2
//   1 x 32000 fp16   16.9, 12.3  23.7, 23.5       128 x 50001 fp32  28.9, 22.4   53, 40
// fp16 with top-p takes 1.1 us for every 1000 logits of a part, and 0.13 for every 1000
// of the row by its counters: rows with large parts are left to these (108 x 120076 in
// two 84 us, by counters 37; 73 x 117468 of mixed settings in three 60, 51; 49 x 78985
// in five 35.5, 40; 32 x 237653, flat ones among them, in eight 46, 100).
int sample_parts(int rows, int vocab) {
    return vocab < kSampleSplit ? 1 : std::max(1, std::min(std::min(kSampleParts, vocab / kSampleShare), kSampleWorkgroups / rows));
}

template <bool FIRST> exq_status sample_call(int bits, const SampleArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.rows * a.split.parts));
    if (bits == 16) hipLaunchKernelGGL((sample_kernel<_Float16, FIRST>), grid, dim3(kSampleThreads), 0, s, a);
    else hipLaunchKernelGGL((sample_kernel<float, FIRST>), grid, dim3(kSampleThreads), 0, s, a);
    return launched("sample launch");
}

}  // namespace

extern "C" size_t exq_sample_workspace_bytes(int rows, int vocab) {
    if (rows < 1 || vocab < 1) return 0;
    const int parts = sample_parts(rows, vocab);
    return parts > 1 ? SampleSplit{nullptr, rows, parts}.bytes() : 0;
}

extern "C" exq_status exq_sample(const void* logits, int bits, int rows, int vocab, int64_t row_stride, const float* u,
                                 const float* temperatures, float temperature, const int32_t* top_ks, int top_k,
                                 const float* top_ps, float top_p, const float* min_ps, float min_p, int32_t* tokens,
                                 float* logprobs, void* workspace, size_t workspace_bytes, void* stream) {
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
    int parts = 1;
    if (workspace) {
        const size_t need = exq_sample_workspace_bytes(rows, vocab);
        if (!aligned(workspace, 16)) return fail(EXQ_ERR_INVALID_ARG, "workspace is misaligned");
        if (workspace_bytes < need) return fail(EXQ_ERR_INVALID_ARG, "workspace of %zu bytes: %zu are needed", workspace_bytes, need);
        if (need && ranges_meet(workspace, need, logits, logits_bytes)) return fail(EXQ_ERR_INVALID_ARG, "workspace overlaps logits");
        for (const auto& x : read)
            if (need && x.p && ranges_meet(workspace, need, x.p, n)) return fail(EXQ_ERR_INVALID_ARG, "workspace overlaps %s", x.name);
        for (const auto& x : written)
            if (need && x.p && ranges_meet(workspace, need, x.p, n)) return fail(EXQ_ERR_INVALID_ARG, "workspace overlaps %s", x.name);
        // (settings for all rows that leave no row to split)
        const bool no_row = (!temperatures && temperature == 0) || (!top_ks && top_k > 0 && top_k < vocab) || (!top_ps && top_p <= 0) ||
                            (!min_ps && min_p > 0 && !top_ps && top_p >= 1);
        if (need && !no_row) parts = sample_parts(rows, vocab);
        if (bits == 16 && vocab > kSampleCountedShare * parts && !top_ps && top_p < 1) parts = 1;
    }
    if ((int64_t)rows * parts * kSampleThreads > kMaxLaunchThreads) return fail(EXQ_ERR_UNSUPPORTED, "%d rows in one call", rows);
    int log2 = 0;
    while ((1 << log2) < vocab) ++log2;
    const SampleArgs a{logits, row_stride, rows, vocab, std::min(51, 63 - log2), u, {temperatures, temperature},
                       {top_ks, top_k}, {top_ps, top_p}, {min_ps, min_p}, tokens, logprobs,
                       {static_cast<uint64_t*>(workspace), rows, parts}};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    exq_status st;
    if (parts > 1 && (st = sample_call<true>(bits, a, s)) != EXQ_OK) return st;
    return sample_call<false>(bits, a, s);
}
