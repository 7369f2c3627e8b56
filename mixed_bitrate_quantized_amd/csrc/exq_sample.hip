// The next token of every row of logits (exq_sample) for gfx950: temperature,
// top-k, top-p and min-p from given random numbers.
//
// With M the row's largest logit and T its temperature, token i weighs
//   w_i = e^{(l_i - M) / T} = 2^t,  t = (l_i - M) log2(e) / T,
// computed in 64 bits and held as a whole number of units of 2^-shift.  Sums of
// whole numbers do not depend on their order, so weights may be added through LDS
// atomics and still give the same token every time; and 2^-45 units keep a border
// between two tokens where the real numbers have it.
//
// One workgroup takes a row; nothing is sorted.  Every filter leaves the tokens
// above a cut: a key (a logit's bits, in order) and how many of those with that key.
//   fp16   a counter in LDS for every key.  The counters say where top-k ends, and
//          with a weight for every key instead of every token (64-bit arithmetic
//          takes 8 cycles an instruction: weights of 131072 tokens take 44 us) what the
//          weights add up to and where top-p ends.
//   fp32   top-k: the k-th largest of the threads' own largest logits is a threshold
//          that at least k logits reach and, with the row dealt out over 1024
//          threads, not many more.  top-p: a histogram of the weights, 64 bins for a
//          power of two.  What may be left goes to LDS, where the cut is found digit by
//          digit of the keys.
// The draw runs over what is left, in LDS, digit by digit of the index, or over
// the row where that is too much: sums of tiles, then the tile that holds it.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "exq_device_common.h"
#include "exq_internal.h"
#include "exq_operand.h"

namespace exq {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int kSampleThreads = 1024, kSampleWaves = kSampleThreads / 64;
constexpr int kSampleList = 4096;             // candidates that LDS holds
constexpr int kSampleEach = kSampleList / kSampleThreads;
constexpr int kDigit = 9;                     // bits looked at together
constexpr int kSampleBins = 2048;             // of a row's histogram
constexpr int kSampleMaxVocabLog2 = 21;
constexpr int kPowers = 256;                  // 2^(i / 256) in LDS
constexpr int kCounters = 1 << 15;            // of 16 bits for each sign

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

// Ordered keys: larger for larger logits; 0 for a NaN or -infinity, which are
// never drawn.  -0 and 0 have one key.
template <class T> struct Logit;
template <> struct Logit<_Float16> {
    typedef h8 vec;
    static constexpr int VEC = 8, BITS = 16, COARSE = 4;   // COARSE: bits of a key below 1/64 of a power of two
    static constexpr bool COUNTED = true;                  // a counter for every key fits LDS
    __device__ static uint32_t key(_Float16 x) {
        uint32_t b = __builtin_bit_cast(uint16_t, x);
        if (b == 0x8000u) b = 0;
        const uint32_t k = b ^ (b & 0x8000u ? 0xFFFFu : 0x8000u);
        return (float)x > -__builtin_huge_valf() ? k : 0u;
    }
    __device__ static float value(uint32_t k) {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(k ^ (k & 0x8000u ? 0x8000u : 0xFFFFu)));
    }
};
template <> struct Logit<float> {
    typedef f4 vec;
    static constexpr int VEC = 4, BITS = 32, COARSE = 17;
    static constexpr bool COUNTED = false;
    __device__ static uint32_t key(float x) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
        return x > -__builtin_huge_valf() ? b ^ (b & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u) : 0u;
    }
    __device__ static float value(uint32_t k) { return __builtin_bit_cast(float, k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu)); }
};

constexpr double kLn2d = 0.69314718055994530942;

// 2^f for |f| <= 1 from its series; the first term left out is below 2^-53 of it
// at 1/2, and 2^-40 at 1.
__device__ __forceinline__ double exp2_series(double f) {
    double p = 1.0;
#pragma unroll
    for (int i = 13; i >= 1; --i) p = __builtin_fma(p, f * (kLn2d / i), 1.0);
    return p;
}

// Weights of a row: 2^(j / 256) from LDS times 2^r, |r| <= 1/512, whose series is cut
// behind r^3: within 2^-45.
struct Weights {
    float topf;
    double top, c;   // largest logit, 256 log2(e) / T; beside an infinity all else weighs nothing
    double scale;    // 2^shift
    double least;    // min-p
    const double* powers;
    __device__ double power(double t) const {   // 2^(t / 256)
#pragma clang fp contract(off)   // the same bits wherever the compiler puts it
        constexpr double a = kLn2d / kPowers;
        t = __builtin_fmax(t, -256.0 * 1000);
        const double n = t + 6755399441055744.0;   // 1.5 * 2^52: rounds t, and leaves it in the sum's low bits
        const double f = t - (n - 6755399441055744.0);
        const int j = (int)(uint32_t)__builtin_bit_cast(uint64_t, n);
        const double near = powers[j & (kPowers - 1)];
        const double q = __builtin_fma(f, __builtin_fma(f, a * a * a / 6, a * a / 2), a);
        const double w = __builtin_fma(near * f, q, near);
        return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, w) + ((uint64_t)(uint32_t)((j >> 8) << 20) << 32));
    }
    __device__ double real(float l) const {   // l: at most the largest
#pragma clang fp contract(off)
        return power(((double)__builtin_fminf(l, __FLT_MAX__) - top) * c);
    }
    // In units, rounded: 2^52 + w * 2^shift has the whole number in its lower bits.
    __device__ uint64_t units(double w) const {
        return __builtin_bit_cast(uint64_t, __builtin_fma(w, scale, 4503599627370496.0)) & 0xFFFFFFFFFFFFFull;
    }
    __device__ uint64_t of(float l) const { return units(real(l)); }
    // Zero below min-p.
    __device__ uint64_t kept(float l) const {
        const double w = real(l);
        return w >= least ? units(w) : 0;
    }
    // ln of its probability among weights of `sum` units
    __device__ float log_of(float l, float temperature, uint64_t sum) const {
        const double z = l == topf ? 0.0 : ((double)l - top) / (double)temperature;
        return (float)(z - log((double)sum / scale));
    }
};

constexpr int kSampleTiles = (1 << kSampleMaxVocabLog2) / 256 + 2;   // at most

struct SampleShared {
    union {
        uint32_t counts[kCounters];      // of magnitude m: positive in the lower half, negative in the upper
        uint64_t list[kSampleList];      // key and index of a candidate
        struct {
            uint64_t sums[kSampleTiles];     // of weights above the cut
            uint32_t equals[kSampleTiles];   // elements at it
        } tile;
    };
    uint64_t bins[kSampleBins];
    double powers[kPowers];
    uint64_t wave[kSampleWaves];
    uint64_t below;
    uint32_t bin, count;
    // counters' sums: for each power of two (and sign), the largest values first
    double block_weight[64];
    uint32_t block_count[64];
    double steps[32][3];   // weights 1, 2, 3 magnitudes behind one, for each power of two
    // a cut found among them
    uint32_t cut_key, cut_above, cut_equal;
    double cut_weight_above, cut_weight, cut_need;
};

// Moves a value within a wave: lanes without a source get 0.
template <int HOW, int ROWS> __device__ __forceinline__ uint64_t moved(uint64_t x) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, HOW, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(x >> 32), HOW, ROWS, 0xF, false);
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t lane_value(uint64_t x, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)x, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), lane);
    return (uint64_t)hi << 32 | lo;
}
struct Sum {
    __device__ static uint64_t of(uint64_t a, uint64_t b) { return a + b; }
};
struct SumReal {
    __device__ static uint64_t of(uint64_t a, uint64_t b) {
        return __builtin_bit_cast(uint64_t, __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b));
    }
};
struct Larger {
    __device__ static uint64_t of(uint64_t a, uint64_t b) { return a > b ? a : b; }
};
// Sums (or largest values) over the lanes up to each one, of 16 and of 64.
template <class Op = Sum> __device__ __forceinline__ uint64_t prefix16(uint64_t x) {
    x = Op::of(x, moved<0x111, 0xF>(x));
    x = Op::of(x, moved<0x112, 0xF>(x));
    x = Op::of(x, moved<0x114, 0xF>(x));
    return Op::of(x, moved<0x118, 0xF>(x));
}
template <class Op = Sum> __device__ __forceinline__ uint64_t prefix64(uint64_t x) {
    x = prefix16<Op>(x);
    x = Op::of(x, moved<0x142, 0xA>(x));   // row 0's to row 1, row 2's to row 3
    return Op::of(x, moved<0x143, 0xC>(x));   // the lower half's to the upper
}
__device__ __forceinline__ double prefix64(double x) {
    return __builtin_bit_cast(double, prefix64<SumReal>(__builtin_bit_cast(uint64_t, x)));
}

// Orders LDS accesses of WAVES waves: all of the workgroup, or one for itself.
template <int WAVES> __device__ __forceinline__ void team_sync() {
    if (WAVES == kSampleWaves) {
        __syncthreads();
    } else {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    }
}

// Over WAVES waves (all of the workgroup, or the one that is left of it): the sum
// of the threads before (with BEFORE), and of all.
template <int WAVES, class Op = Sum, bool BEFORE = false>
__device__ __forceinline__ uint64_t reduce(SampleShared& s, uint64_t x, uint64_t* before = nullptr) {
    static_assert(WAVES == 1 || WAVES == 16, "a row of lanes adds up the waves");
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const uint64_t sums = prefix64<Op>(x);
    if (WAVES == 1) {
        if (BEFORE) *before = sums - x;
        return lane_value(sums, 63);
    }
    __syncthreads();
    if (lane == 63) s.wave[wave] = sums;
    __syncthreads();
    const uint64_t waves = prefix16<Op>(s.wave[lane & 15]);
    if (BEFORE) *before = sums - x + (wave ? lane_value(waves, wave - 1) : 0);
    return lane_value(waves, 15);
}

// The bin of 64 PER that takes the running sum from the first one to `need`
// or more, and the sum below it; by one wave, for all after a barrier.
template <int WAVES, int PER> __device__ __forceinline__ void find_bin(SampleShared& s, uint64_t need) {
    team_sync<WAVES>();
    if (threadIdx.x < 64) {
        uint64_t x[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            x[i] = s.bins[PER * threadIdx.x + i];
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
    team_sync<WAVES>();
}

__device__ __forceinline__ void add_to_bin(SampleShared& s, uint32_t bin, uint64_t amount) {
    atomicAdd(reinterpret_cast<unsigned long long*>(&s.bins[bin]), (unsigned long long)amount);
}

// The smallest D below 2^bits with a sum of amounts of d <= D of `need` or more
// (which all d reach), digit by digit; `below`: the sum of the smaller ones.
// source(f) calls f(d, amount) for the thread's elements.
template <int WAVES, class S>
__device__ __forceinline__ uint32_t select(SampleShared& s, int bits, uint64_t need, uint64_t& below, S&& source) {
    uint32_t value = 0;
    below = 0;
    for (int high = bits, low; high > 0; high = low) {
        low = max(high - kDigit, 0);
        team_sync<WAVES>();
#pragma unroll
        for (int i = 0; i < 1 << kDigit; i += 64 * WAVES)
            if (WAVES == 1 || threadIdx.x < 1 << kDigit) s.bins[threadIdx.x + i] = 0;
        team_sync<WAVES>();
        const bool first = high == bits;
        source([&](uint32_t d, uint64_t amount) {
            const uint32_t digit = d >> low;
            if ((first || (digit ^ (value >> low)) >> (high - low) == 0) && amount)
                add_to_bin(s, digit & ((1u << (high - low)) - 1), amount);
        });
        find_bin<WAVES, (1 << kDigit) / 64>(s, need - below);
        value |= s.bin << low;
        below += s.below;
    }
    return value;
}

template <class T> __device__ __forceinline__ int head_elements(const T* row, int vocab) {
    return min(vocab, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T));
}

// each(vector, index) for the thread's vectors of the row, AHEAD loaded at a time,
// and one(value, index) for the ends of the row, fewer than a vector each.
template <class T, int AHEAD, class F, class G>
__device__ __forceinline__ void for_vectors(const T* row, int vocab, F&& each, G&& one) {
    typedef typename Logit<T>::vec vec;
    constexpr int VEC = Logit<T>::VEC;
    const int t = threadIdx.x, head = head_elements(row, vocab), vecs = (vocab - head) / VEC, tail = head + vecs * VEC;
    const EXQ_GLOBAL vec* body = gptr<vec>(row + head);
    for (int j = t; j < vecs; j += AHEAD * kSampleThreads) {
        vec x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) x[i] = j + i * kSampleThreads < vecs ? body[j + i * kSampleThreads] : vec{};
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (j + i * kSampleThreads < vecs) each(x[i], head + (j + i * kSampleThreads) * VEC);
    }
    const int ends = head + vocab - tail;
    if (t < ends) {
        const int i = t < head ? t : tail + t - head;
        one(row[i], i);
    }
}

// f(index, value) for the thread's elements of the row.
template <class T, int AHEAD, class F> __device__ __forceinline__ void for_row(const T* row, int vocab, F&& f) {
    for_vectors<T, AHEAD>(row, vocab, [&](const typename Logit<T>::vec& x, int i) {
#pragma unroll
        for (int e = 0; e < Logit<T>::VEC; ++e) f(i + e, x[e]);
    }, [&](T x, int i) { f(i, x); });
}

// What the filters left: keys above `key`, and of those with it the first `quota`.
struct Cut {
    uint32_t key, quota;
};

// ------------------------------------------------------- counters of fp16 keys

// Counts a row and returns the thread's largest logit.
__device__ __forceinline__ float count_row(SampleShared& s, const _Float16* row, int vocab) {
    u4v* zero = reinterpret_cast<u4v*>(s.counts);
#pragma unroll
    for (int i = 0; i < kCounters / 4; i += kSampleThreads) zero[threadIdx.x + i] = u4v{0, 0, 0, 0};
    __syncthreads();
    const _Float16 lowest = -(_Float16)__builtin_huge_valf();
    h8 most = {lowest, lowest, lowest, lowest, lowest, lowest, lowest, lowest};
    const auto count = [&](uint32_t bits) {   // of the lower half
        atomicAdd(&s.counts[bits & 0x7FFFu], bits & 0x8000u ? 0x10000u : 1u);
    };
    for_vectors<_Float16, 8>(row, vocab, [&](const h8& x, int) {
        most = __builtin_elementwise_max(most, x);
        const u4v bits = __builtin_bit_cast(u4v, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            count(bits[i]);
            count(bits[i] >> 16);
        }
    }, [&](_Float16 x, int) {
        most[0] = __builtin_elementwise_max(most[0], x);
        count(__builtin_bit_cast(uint16_t, x));
    });
    float top = (float)most[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, (float)most[i]);
    return top;
}

// Four neighbouring magnitudes of one sign, from the largest logit to the smallest.
struct Four {
    uint32_t n[4], key[4], all;
    double w[4];
};

// The lane's of 256: magnitudes of power of two `block`, part `part` of 4.  Largest
// logits come first: with positive ones the upper lanes' magnitudes in turn.
template <bool NEGATIVE> __device__ __forceinline__ Four four_of(const SampleShared& s, int block, int part) {
    const int lane = threadIdx.x & 63, m0 = 1024 * block + 256 * (NEGATIVE ? part : 3 - part) + 4 * (NEGATIVE ? lane : 63 - lane);
    const u4v c = *reinterpret_cast<const u4v*>(&s.counts[m0]);
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

// Their weights, and what the counted ones add up to.  Neighbours' weights have
// one ratio within a power of two.
__device__ __forceinline__ double weigh(const SampleShared& s, const Weights& w, uint32_t top_key, int block, Four& x) {
    x.w[0] = x.w[1] = x.w[2] = x.w[3] = 0;
    if (x.all == 0) return 0.0;
    if (x.key[0] <= top_key) {
        x.w[0] = w.real(Logit<_Float16>::value(x.key[0]));
#pragma unroll
        for (int e = 1; e < 4; ++e) x.w[e] = x.w[0] * s.steps[block][e - 1];
    } else {   // some, not counted, lie above the largest logit
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (x.key[e] <= top_key) x.w[e] = w.real(Logit<_Float16>::value(x.key[e]));
    }
    return __builtin_fma(x.n[3], x.w[3], __builtin_fma(x.n[2], x.w[2], __builtin_fma(x.n[1], x.w[1], x.n[0] * x.w[0])));
}

// Adds the counters up by power of two and sign, their weights too if asked for.
// The number of logits that may be drawn; -1: a counter overflowed (65536 equal ones).
__device__ __forceinline__ int sum_counters(SampleShared& s, const Weights& w, uint32_t top_key, bool weights, int vocab) {
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t / 64), lane = t & 63;
    if (weights && t < 32 * 3)   // neighbours of a power of two lie 2^(block - 25) apart
        s.steps[t / 3][t % 3] = w.power(-(1 + t % 3) * __builtin_ldexp(w.c, max(t / 3, 1) - 25));
    __syncthreads();
    uint64_t all = 0;
#pragma unroll 1
    for (int block = wave; block < 32; block += kSampleWaves) {
        uint32_t n[2] = {0, 0};
        double sum[2] = {0, 0};
#pragma unroll 1
        for (int part = 0; part < 4; ++part) {
            Four x = four_of<false>(s, block, part);
            n[0] += x.all;
            if (weights) sum[0] += weigh(s, w, top_key, block, x);
            x = four_of<true>(s, block, part);
            n[1] += x.all;
            if (weights) sum[1] += weigh(s, w, top_key, block, x);
        }
        all += n[0] + n[1];
#pragma unroll
        for (int sign = 0; sign < 2; ++sign) {
            const uint32_t count = (uint32_t)prefix64((uint64_t)n[sign]);
            const double weight = weights ? prefix64(sum[sign]) : 0.0;
            if (lane == 63) {
                s.block_count[sign ? 32 + block : 31 - block] = count;
                s.block_weight[sign ? 32 + block : 31 - block] = weight;
            }
        }
    }
    // -infinity and NaN were not counted above
    uint64_t rest = 0;
    for (int m = 0x7C00 + t; m < kCounters; m += kSampleThreads) rest += (s.counts[m] >> 16) + (m > 0x7C00 ? s.counts[m] & 0xFFFFu : 0);
    const uint64_t both = reduce<kSampleWaves>(s, all | rest << 32);
    return (both & 0xFFFFFFFFu) + (both >> 32) == (uint64_t)vocab ? (int)(uint32_t)both : -1;
}

// Where the running sum of counts, or weights, reaches `need` (with `share`: that
// share of all weights): into s.cut_*.
__device__ __forceinline__ void find_key(SampleShared& s, const Weights& w, uint32_t top_key, bool counts, double need, bool weights,
                                         bool share) {
    __syncthreads();
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        const auto at_lane = [](double x, int i) { return __builtin_bit_cast(double, lane_value(__builtin_bit_cast(uint64_t, x), i)); };
        const double n = s.block_count[lane], weight = s.block_weight[lane];
        const double n_to = prefix64(n), w_to = prefix64(weight);
        if (share) need *= at_lane(w_to, 63);
        // (the last block that holds anything, if rounding kept the sum below)
        const uint64_t reach = __ballot((counts ? n_to : w_to) >= need && n > 0), any = __ballot(n > 0);
        const int at = reach ? __builtin_ctzll(reach) : 63 - __builtin_clzll(any);
        double n_before = at_lane(n_to - n, at), w_before = at_lane(w_to - weight, at);
        const int block = at >= 32 ? at - 32 : 31 - at;
#pragma unroll 1
        for (int part = 0; part < 4; ++part) {
            Four x = at >= 32 ? four_of<true>(s, block, part) : four_of<false>(s, block, part);
            const double here = x.all, here_w = weights ? weigh(s, w, top_key, block, x) : 0.0;
            const double here_to = prefix64(here), here_w_to = prefix64(here_w);
            const uint64_t some = __ballot(x.all != 0);
            const uint64_t found = __ballot(x.all != 0 && (counts ? n_before + here_to : w_before + here_w_to) >= need);
            // the lane that reaches it; so far, the last one that holds anything
            if (some && lane == (found ? __builtin_ctzll(found) : 63 - __builtin_clzll(some))) {
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
            if (lane == 0) s.cut_need = need;
            if (found) break;
            n_before += at_lane(here_to, 63);
            w_before += at_lane(here_w_to, 63);
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- candidates

// What ends a row on its list of `count` candidates, by WAVES waves.
struct Finish {
    int count, vocab;
    uint32_t top_key;
    int key_bits, index_bits;
    int top_k;           // 0: done
    float top_p;         // 1 or more: done
    uint64_t share;      // what top-p needs, if it is of more than the list; else 0
    Cut cut;
    float u, temperature;
};

__device__ __forceinline__ uint64_t share_of(float top_p, uint64_t total) {   // what top-p needs of it
    return std::min<uint64_t>(std::max<uint64_t>((uint64_t)__builtin_ceil((double)top_p * (double)total), 1), total);
}
__device__ __forceinline__ uint64_t target_of(float u, uint64_t total) {
    return std::min<uint64_t>((uint64_t)((double)u * (double)total), total - 1);
}

template <class T, int WAVES, class A>
__device__ __forceinline__ void finish(SampleShared& s, const Weights& w, Finish f, A&& answer) {
    typedef Logit<T> L;
    constexpr int N = 64 * WAVES;
    uint32_t keys[kSampleEach], at[kSampleEach];
    uint64_t ws[kSampleEach];
#pragma unroll
    for (int i = 0; i < kSampleEach; ++i) {
        keys[i] = at[i] = 0;
        ws[i] = 0;
        if ((int)threadIdx.x + i * N < f.count) {
            const uint64_t x = s.list[threadIdx.x + i * N];
            keys[i] = (uint32_t)(x >> 32);
            at[i] = (uint32_t)x;
            ws[i] = w.of(L::value(keys[i]));
        }
    }
    const auto each = [&](auto&& g) {
#pragma unroll
        for (int i = 0; i < kSampleEach; ++i)
            if (i * N < f.count && keys[i]) g(keys[i], at[i], ws[i]);
    };
    uint64_t below;
#pragma unroll 1
    for (int filter = f.top_k ? 0 : 1; filter < (f.top_p < 1.0f ? 2 : 1); ++filter) {
        const bool counts = filter == 0;
        uint64_t all = 0;
        each([&](uint32_t k, uint32_t, uint64_t x) { all += k < f.cut.key ? 0 : counts ? 1 : k > f.cut.key ? x : 0; });
        all = reduce<WAVES>(s, all);
        if (!counts && f.cut.key) all += f.cut.quota * w.of(L::value(f.cut.key));
        const uint64_t need = counts ? (uint64_t)f.top_k : f.share ? f.share : share_of(f.top_p, all);
        if (need >= all) continue;
        const uint32_t key = f.top_key - select<WAVES>(s, f.key_bits, need, below, [&](auto&& g) {
            each([&](uint32_t k, uint32_t, uint64_t x) {
                if (k >= f.cut.key) g(f.top_key - k, counts ? 1 : x);
            });
        });
        const uint64_t one = counts ? 1 : w.of(L::value(key));
        f.cut = Cut{key, (uint32_t)((need - below + one - 1) / one)};
    }
    // of those at the cut the first ones
    uint32_t last = 0xFFFFFFFFu;
    uint64_t equal = 0;
    each([&](uint32_t k, uint32_t, uint64_t) { equal += k == f.cut.key; });
    if (reduce<WAVES>(s, equal) > f.cut.quota)
        last = select<WAVES>(s, f.index_bits, f.cut.quota, below, [&](auto&& g) {
            each([&](uint32_t k, uint32_t i, uint64_t) {
                if (k == f.cut.key) g(i, 1);
            });
        });
    uint64_t sum = 0;
    each([&](uint32_t k, uint32_t i, uint64_t& x) {
        const bool in = k > f.cut.key || (k == f.cut.key && i <= last);
        x = in ? w.kept(L::value(k)) : 0;
        sum += x;
    });
    sum = reduce<WAVES>(s, sum);
    // the draw: indices in ascending order
    const uint32_t token = select<WAVES>(s, f.index_bits, target_of(f.u, sum) + 1, below, [&](auto&& g) {
        each([&](uint32_t, uint32_t i, uint64_t x) { g(i, x); });
    });
    each([&](uint32_t k, uint32_t i, uint64_t) {
        if (i == token) answer((int)token, w.log_of(L::value(k), f.temperature, sum));
    });
}

// -------------------------------------------------------------------- kernel

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
    const bool first_only = temperature == 0.0f || top_k == 1 || top_p <= 0.0f || min_p > 1.0f;
    const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.0f;
    if (t < kPowers) s.powers[t] = exp2_series((double)t / kPowers);
    if (t == 0) s.bin = s.below = 0;

    // the largest logit
    bool counted = L::COUNTED && !first_only && (by_k || by_p);
    uint64_t best = 0;
    uint32_t mine = 0;   // the thread's own
    if constexpr (L::COUNTED) {
        if (counted) best = (uint64_t)L::key((_Float16)count_row(s, row, a.vocab)) << 32;
    }
    if (!counted) {   // and its lowest index
        for_row<T, 4>(row, a.vocab, [&](int i, T x) {
            const uint64_t it = (uint64_t)L::key(x) << 32 | (uint32_t)~i;
            if (it >> 32) best = std::max(best, it);
        });
        mine = (uint32_t)(best >> 32);
    }
    best = reduce<kSampleWaves, Larger>(s, best);
    if (best == 0) {   // nothing that may be drawn
        if (t == 0) answer(-1, __builtin_nanf(""));
        return;
    }
    if (first_only) {
        if (t == 0) answer((int)~(uint32_t)best, 0.0f);
        return;
    }
    const uint32_t top_key = (uint32_t)(best >> 32);
    const float topf = L::value(top_key), finite_top = __builtin_fminf(topf, __FLT_MAX__);
    const Weights w{topf, (double)finite_top, topf > __FLT_MAX__ ? 1e300 : kPowers * 1.4426950408889634074 / (double)temperature,
                    (double)(1ull << a.shift), min_p, s.powers};
    Finish f{0, a.vocab, top_key, L::BITS, a.vocab > 1 << 2 * kDigit ? kSampleMaxVocabLog2 : 2 * kDigit, 0, 1.0f, 0,
             Cut{0, 0xFFFFFFFFu}, u, temperature};

    // Elements that want(key, value) asks for, into the list.
    const auto collect = [&](auto&& want) {
        __syncthreads();
        if (t == 0) s.count = 0;
        __syncthreads();
        for_row<T, 4>(row, a.vocab, [&](int i, T x) {
            const uint32_t k = L::key(x);
            if (k && want(k, x)) {
                const uint32_t at = atomicAdd(&s.count, 1u);
                if (at < kSampleList) s.list[at] = (uint64_t)k << 32 | (uint32_t)i;
            }
        });
        __syncthreads();
        return (int)std::min<uint32_t>(s.count, 0x7FFFFFFFu);
    };

    if (by_k || by_p) {
        bool held = false;   // whether the list holds all that the filters can leave
        if constexpr (L::COUNTED) {
            const int some = counted ? sum_counters(s, w, top_key, by_p, a.vocab) : -1;
            counted = some >= 0;
            if (counted) {
                uint32_t kept = 0;   // at the cut or above
                if (by_k && some > top_k) {
                    find_key(s, w, top_key, true, (double)top_k, by_p, false);
                    f.cut = Cut{s.cut_key, (uint32_t)top_k - s.cut_above};
                    kept = s.cut_above + s.cut_equal;
                }
                if (by_p) {
                    const bool cut = f.cut.key != 0;
                    find_key(s, w, top_key, false, (double)top_p * (cut ? s.cut_weight_above + f.cut.quota * s.cut_weight : 1.0), true, !cut);
                    const double ties = __builtin_ceil((s.cut_need - s.cut_weight_above) / s.cut_weight);
                    uint32_t quota = ties < 1.0 ? 1u : ties > (double)s.cut_equal ? s.cut_equal : (uint32_t)ties;
                    if (f.cut.key == s.cut_key) quota = std::min(quota, f.cut.quota);
                    f.cut = Cut{s.cut_key, quota};
                    kept = s.cut_above + s.cut_equal;
                }
                if (f.cut.key && kept <= kSampleList) {
                    f.count = collect([&](uint32_t k, T) { return k >= f.cut.key; });
                    held = true;
                }
            } else {   // an overflow: the threads' largest logits for what follows
                for_row<T, 4>(row, a.vocab, [&](int, T x) { mine = std::max(mine, L::key(x)); });
            }
        }
        if (!counted) {
            uint64_t below;
            if (by_k) {
                // a threshold that top_k threads' largest logits reach, to 1/64 of a power of two
                const auto coarse = [&](uint32_t k) { return min((top_key >> L::COARSE) - (k >> L::COARSE), (1u << kDigit) - 1); };
                const uint64_t want = std::min<uint64_t>(top_k, reduce<kSampleWaves>(s, mine ? 1 : 0));
                const uint32_t least = select<kSampleWaves>(s, kDigit, want, below, [&](auto&& g) {
                    if (mine) g(coarse(mine), 1);
                });
                f.count = collect([&](uint32_t k, T) { return coarse(k) <= least; });
                held = f.count <= kSampleList && f.count >= top_k;
                f.top_k = top_k;
                f.top_p = top_p;
                // the keys lie that near the top, or anywhere from the last bin on
                if (least < (1u << kDigit) - 1) f.key_bits = L::COARSE + kDigit;
            }
#pragma unroll 1
            for (int filter = by_k ? 0 : 1; !held && filter < (by_p ? 2 : 1); ++filter) {
                const bool counts = filter == 0;
                // 64 bins for one of the logits, or for a power of two of the weights
                const float rate = counts ? 64.0f : __builtin_fminf((float)(w.c * (64.0 / kPowers)), 1e30f);
                const auto bin_of = [&](float l) {
                    const float d = (finite_top - __builtin_fminf(l, __FLT_MAX__)) * rate;
                    return d < (float)(kSampleBins - 1) ? (int)d : kSampleBins - 1;
                };
                __syncthreads();
                for (int i = t; i < kSampleBins; i += kSampleThreads) s.bins[i] = 0;
                __syncthreads();
                for_row<T, 2>(row, a.vocab, [&](int, T x) {
                    const uint32_t k = L::key(x);
                    if (k && k >= f.cut.key) {
                        const uint64_t amount = counts ? 1 : k > f.cut.key ? w.of((float)x) : 0;
                        if (amount) add_to_bin(s, (uint32_t)bin_of((float)x), amount);
                    }
                });
                if (!counts && f.cut.key && t == 0) {
                    const float l = L::value(f.cut.key);
                    add_to_bin(s, (uint32_t)bin_of(l), f.cut.quota * w.of(l));
                }
                __syncthreads();
                uint64_t all = 0;
                for (int i = t; i < kSampleBins; i += kSampleThreads) all += s.bins[i];
                all = reduce<kSampleWaves>(s, all);
                const uint64_t need = counts ? (uint64_t)top_k : share_of(top_p, all);
                if (need >= all) continue;
                find_bin<kSampleWaves, kSampleBins / 64>(s, need);
                const int bin = (int)s.bin;
                const uint64_t before = s.below;
                if (!counts) {   // all that is left fits the list?
                    f.count = collect([&](uint32_t k, T x) { return k >= f.cut.key && bin_of((float)x) <= bin; });
                    if (f.count <= kSampleList) {
                        held = true;
                        f.top_k = 0;
                        f.top_p = top_p;
                        f.share = need;
                        f.key_bits = L::BITS;
                        break;
                    }
                }
                const int count = collect([&](uint32_t k, T x) { return k >= f.cut.key && bin_of((float)x) == bin; });
                uint64_t skipped;
                uint32_t d;
                if (count <= kSampleList) {
                    d = select<kSampleWaves>(s, L::BITS, need - before, skipped, [&](auto&& g) {
#pragma unroll 1
                        for (int i = t; i < count; i += kSampleThreads) {
                            const uint32_t k = (uint32_t)(s.list[i] >> 32);
                            g(top_key - k, counts ? 1 : w.of(L::value(k)));
                        }
                    });
                    skipped += before;
                } else {   // equal or nearly equal ones: over the row again
                    d = select<kSampleWaves>(s, L::BITS, need, skipped, [&](auto&& g) {
                        for_row<T, 1>(row, a.vocab, [&](int, T x) {
                            const uint32_t k = L::key(x);
                            if (k && k >= f.cut.key) g(top_key - k, counts ? 1 : w.of((float)x));
                        });
                    });
                }
                const uint64_t one = counts ? 1 : w.of(L::value(top_key - d));
                f.cut = Cut{top_key - d, (uint32_t)((need - skipped + one - 1) / one)};
            }
        }
        if (held) {
            if (f.count > 64 * kSampleEach) {
                finish<T, kSampleWaves>(s, w, f, answer);
            } else if (t < 64) {
                finish<T, 1>(s, w, f, answer);
            }
            return;
        }
        __syncthreads();
    }

    // the draw over the whole row: sums of tiles, then the tile that holds it
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
    const uint64_t one = f.cut.key ? w.kept(L::value(f.cut.key)) : 0;   // of those at the cut
    for (int tile = t / 64; tile < tiles; tile += kSampleWaves) {
        const Span at = span(tile);
        uint64_t sum = 0;
        uint32_t equal = 0;
        const auto add = [&](T l) {
            const uint32_t k = L::key(l);
            equal += k && k == f.cut.key;
            if (k > f.cut.key) sum += w.kept((float)l);
        };
        if (at.n == L::VEC) {
            const typename L::vec v = *gptr<typename L::vec>(row + at.first);
#pragma unroll
            for (int e = 0; e < L::VEC; ++e) add(v[e]);
        } else if (at.n) {
            add(row[at.first]);
        }
        sum = prefix64(sum);
        const uint32_t equals = (uint32_t)prefix64((uint64_t)equal);
        if (lane == 63) {
            s.tile.sums[tile] = sum;
            s.tile.equals[tile] = equals;
        }
    }
    __syncthreads();
    const int per = (tiles + kSampleThreads - 1) / kSampleThreads, begin = std::min(tiles, t * per), end = std::min(tiles, (t + 1) * per);
    uint64_t equal = 0, equal_before, sum = 0, before;
    for (int i = begin; i < end; ++i) equal += s.tile.equals[i];
    reduce<kSampleWaves, Sum, true>(s, equal, &equal_before);
    const auto taken = [&](uint64_t from, uint64_t n) {   // of n at the cut behind `from` others
        return from >= f.cut.quota ? 0 : std::min<uint64_t>(n, f.cut.quota - from);
    };
    equal = equal_before;
    for (int i = begin; i < end; ++i) {
        sum += s.tile.sums[i] + taken(equal, s.tile.equals[i]) * one;
        equal += s.tile.equals[i];
    }
    const uint64_t total = reduce<kSampleWaves, Sum, true>(s, sum, &before), target = target_of(u, total);
    if (before <= target && target < before + sum) {
        equal = equal_before;
        for (int i = begin; i < end; ++i) {
            const uint64_t here = s.tile.sums[i] + taken(equal, s.tile.equals[i]) * one;
            if (target < before + here) {
                s.bin = i;
                s.below = before;
                s.count = (uint32_t)equal;
                break;
            }
            before += here;
            equal += s.tile.equals[i];
        }
    }
    __syncthreads();
    if (t >= 64) return;
    const Span at = span((int)s.bin);
    uint32_t lane_equal = 0;
#pragma unroll 1
    for (int e = 0; e < at.n; ++e) lane_equal += L::key(row[at.first + e]) == f.cut.key && f.cut.key;
    const uint32_t equal_first = s.count + (uint32_t)prefix64((uint64_t)lane_equal) - lane_equal;
    uint64_t lane_sum = 0, reached = 0;
    // once for the lane's sum, and once for the element
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
        uint32_t seen = equal_first;
        uint64_t sums = 0;
#pragma unroll 1
        for (int e = 0; e < at.n; ++e) {
            const T l = row[at.first + e];
            const uint32_t k = L::key(l);
            uint64_t x = 0;
            if (k > f.cut.key) x = w.kept((float)l);
            else if (k && k == f.cut.key) x = seen++ < f.cut.quota ? one : 0;
            sums += x;
            if (round && target < reached + sums) {
                answer(at.first + e, w.log_of((float)l, temperature, total));
                break;
            }
        }
        if (round) break;
        lane_sum = sums;
        reached = s.below + prefix64(lane_sum) - lane_sum;
        if (!(reached <= target && target < reached + lane_sum)) break;
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
