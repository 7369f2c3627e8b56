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
// by digit of their indices.  Where the cut lies below them (nearly flat rows, or a
// top-k in the thousands), a histogram of the whole row narrows it to one bin.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "exq_device_common.h"
#include "exq_internal.h"
#include "exq_operand.h"

namespace exq {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int kSampleThreads = 1024, kSampleWaves = kSampleThreads / 64;
constexpr int kSampleList = 4096;             // candidates that LDS holds
constexpr int kSampleWant = 900;               // threads' largest logits that bound top-p's candidates
constexpr int kSampleEach = kSampleList / kSampleThreads;
constexpr int kDigit = 9;                     // bits looked at together
constexpr int kSampleBins = 2048;             // of a row's histogram
constexpr int kSampleMaxVocabLog2 = 21;
constexpr int kPowers = 256;                  // 2^(i / 256) in LDS

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
    __device__ double real(float l) const {
#pragma clang fp contract(off)   // the same bits wherever the compiler puts it
        constexpr double a = kLn2d / kPowers;
        const double t = __builtin_fmax(((double)__builtin_fminf(l, __FLT_MAX__) - top) * c, -256.0 * 1000);
        const double n = t + 6755399441055744.0;   // 1.5 * 2^52: rounds t, and leaves it in the sum's low bits
        const double f = t - (n - 6755399441055744.0);
        const int j = (int)(uint32_t)__builtin_bit_cast(uint64_t, n);
        const double power = powers[j & (kPowers - 1)];
        const double q = __builtin_fma(f, __builtin_fma(f, a * a * a / 6, a * a / 2), a);
        const double w = __builtin_fma(power * f, q, power);
        return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, w) + ((uint64_t)(uint32_t)((j >> 8) << 20) << 32));
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

struct SampleShared {
    union {
        uint64_t list[kSampleList];                             // key and index of a candidate
        uint64_t tiles[(1 << kSampleMaxVocabLog2) / 256 + 2];   // sums of weights
    };
    uint64_t bins[kSampleBins];
    double powers[kPowers];
    uint64_t wave[kSampleWaves];
    uint64_t below;
    uint32_t bin, count;
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

// Over the workgroup: the sum of the threads before (with BEFORE), and of all.
template <class Op = Sum, bool BEFORE = false>
__device__ __forceinline__ uint64_t block_reduce(SampleShared& s, uint64_t x, uint64_t* before = nullptr) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
    const uint64_t sums = prefix64<Op>(x);
    __syncthreads();
    if (lane == 63) s.wave[wave] = sums;
    __syncthreads();
    const uint64_t waves = prefix16<Op>(s.wave[lane & 15]);
    if (BEFORE) *before = sums - x + (wave ? lane_value(waves, wave - 1) : 0);
    return lane_value(waves, 15);
}
static_assert(kSampleWaves == 16, "a row of lanes adds up the waves");

// The bin of 64 PER that takes the running sum from the first one to `need`
// or more, and the sum below it; by one wave, for all after a barrier.
template <int PER> __device__ __forceinline__ void find_bin(SampleShared& s, uint64_t need) {
    __syncthreads();
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
    __syncthreads();
}

__device__ __forceinline__ void add_to_bin(SampleShared& s, uint32_t bin, uint64_t amount) {
    atomicAdd(reinterpret_cast<unsigned long long*>(&s.bins[bin]), (unsigned long long)amount);
}

// The smallest D below 2^bits with a sum of amounts of d <= D of `need` or more
// (which all d reach), digit by digit; `below`: the sum of the smaller ones.
// source(f) calls f(d, amount) for the thread's elements.
template <class S>
__device__ __forceinline__ uint32_t select(SampleShared& s, int bits, uint64_t need, uint64_t& below, S&& source) {
    uint32_t value = 0;
    below = 0;
    for (int high = bits, low; high > 0; high = low) {
        low = max(high - kDigit, 0);
        __syncthreads();
        if (threadIdx.x < 1 << kDigit) s.bins[threadIdx.x] = 0;
        __syncthreads();
        const bool first = high == bits;
        source([&](uint32_t d, uint64_t amount) {
            const uint32_t digit = d >> low;
            if ((first || (digit ^ (value >> low)) >> (high - low) == 0) && amount)
                add_to_bin(s, digit & ((1u << (high - low)) - 1), amount);
        });
        find_bin<(1 << kDigit) / 64>(s, need - below);
        value |= s.bin << low;
        below += s.below;
    }
    return value;
}
__device__ __forceinline__ int bits_of(uint32_t x) { return x ? 32 - __builtin_clz(x) : 0; }

template <class T> __device__ __forceinline__ int head_elements(const T* row, int vocab) {
    return min(vocab, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T));
}

// f(index, value) for the thread's elements of the row, AHEAD vectors loaded at
// a time.
template <class T, int AHEAD, class F> __device__ __forceinline__ void for_row(const T* row, int vocab, F&& f) {
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
            if (j + i * kSampleThreads < vecs)
#pragma unroll
                for (int e = 0; e < VEC; ++e) f(head + (j + i * kSampleThreads) * VEC + e, x[i][e]);
    }
    // the row's ends, fewer than a vector each
    const int ends = head + vocab - tail;
    if (t < ends) {
        const int i = t < head ? t : tail + t - head;
        f(i, row[i]);
    }
}

// What the filters left: keys above `key`, and of those equal the indices up to
// `index`.
struct Cut {
    uint32_t key, index;
    __device__ bool keeps(uint32_t k, uint32_t i) const { return k > key || (k == key && i <= index); }
};

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
    for_row<T, 4>(row, a.vocab, [&](int i, T x) {
        const uint64_t it = (uint64_t)L::key(x) << 32 | (uint32_t)~i;
        if (it >> 32) best = std::max(best, it);
    });
    const uint32_t mine = (uint32_t)(best >> 32);
    if (t < kPowers) s.powers[t] = exp2_series((double)t / kPowers);
    if (t == 0) s.bin = s.below = 0;
    best = block_reduce<Larger>(s, best);
    if (best == 0) {   // nothing that may be drawn
        if (t == 0) answer(-1, __builtin_nanf(""));
        return;
    }
    if (temperature == 0.0f || top_k == 1 || top_p <= 0.0f || min_p > 1.0f) {
        if (t == 0) answer((int)~(uint32_t)best, 0.0f);
        return;
    }
    const uint32_t top_key = (uint32_t)(best >> 32);
    const float topf = L::value(top_key), finite_top = __builtin_fminf(topf, __FLT_MAX__);
    const Weights w{topf, (double)finite_top, topf > __FLT_MAX__ ? 1e300 : kPowers * 1.4426950408889634074 / (double)temperature,
                    (double)(1ull << a.shift), min_p, s.powers};
    const int index_bits = a.vocab > 1 << 2 * kDigit ? kSampleMaxVocabLog2 : 2 * kDigit;
    Cut cut{0, 0xFFFFFFFFu};

    // Elements that want(key, value) asks for, and the cut keeps, into the list.
    const auto collect = [&](auto&& want) {
        __syncthreads();
        if (t == 0) s.count = 0;
        __syncthreads();
        for_row<T, 2>(row, a.vocab, [&](int i, T x) {
            const uint32_t k = L::key(x);
            if (k && want(k, x) && cut.keeps(k, (uint32_t)i)) {
                const uint32_t at = atomicAdd(&s.count, 1u);
                if (at < kSampleList) s.list[at] = (uint64_t)k << 32 | (uint32_t)i;
            }
        });
        __syncthreads();
        return (int)std::min<uint32_t>(s.count, 0x7FFFFFFFu);
    };

    const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.0f;
    if (by_k || by_p) {
        uint64_t below;
        // a threshold that `want` threads' largest logits reach, to 1/64 of a power of two
        const auto coarse = [&](uint32_t k) { return min((top_key >> L::COARSE) - (k >> L::COARSE), (1u << kDigit) - 1); };
        const uint64_t threads = block_reduce(s, mine ? 1 : 0);
        const uint64_t want = std::min<uint64_t>(by_k ? (uint64_t)top_k : kSampleWant, threads);
        const uint32_t least = select(s, kDigit, want, below, [&](auto&& f) {
            if (mine) f(coarse(mine), 1);
        });
        double thread_sum = 0;
        int count = collect([&](uint32_t k, T l) {
            if (!by_k) thread_sum += w.real((float)l);
            return coarse(k) <= least;
        });
        const auto share = [&](uint64_t total) {   // what top-p needs of it
            return std::min<uint64_t>(std::max<uint64_t>((uint64_t)__builtin_ceil((double)top_p * (double)total), 1), total);
        };
        // top-p's share of the whole row
        const uint64_t row_share = by_k ? 0 : share(block_reduce(s, (uint64_t)__builtin_rint(thread_sum * w.scale)));

        // the thread's candidates
        uint32_t keys[kSampleEach], at[kSampleEach];
        uint64_t ws[kSampleEach];
        const auto load = [&] {
#pragma unroll
            for (int i = 0; i < kSampleEach; ++i) {
                keys[i] = at[i] = 0;
                ws[i] = 0;
                if (t + i * kSampleThreads < count) {
                    const uint64_t x = s.list[t + i * kSampleThreads];
                    keys[i] = (uint32_t)(x >> 32);
                    at[i] = (uint32_t)x;
                    ws[i] = w.of(L::value(keys[i]));
                }
            }
        };
        const auto each = [&](auto&& f) {
#pragma unroll
            for (int i = 0; i < kSampleEach; ++i)
                if (i * kSampleThreads < count && keys[i]) f(keys[i], at[i], ws[i]);
        };
        // Whether the candidates hold what the filters leave: else they are found anew, around each filter's cut.
        bool held = count <= kSampleList && (!by_k || count >= top_k);
        if (held) {
            load();
            if (!by_k) {
                uint64_t here = 0;
                each([&](uint32_t, uint32_t, uint64_t x) { here += x; });
                held = block_reduce(s, here) >= row_share;
            }
        }
        // their keys lie that near the top, or anywhere from the last bin on
        const int held_bits = least < (1u << kDigit) - 1 ? L::COARSE + kDigit : L::BITS;

#pragma unroll 1
        for (int filter = by_k ? 0 : 1; filter < (by_p ? 2 : 1); ++filter) {
            const bool counts = filter == 0;
            uint64_t need, all = 0;   // of those in the cut (or in the bin that holds the next one)
            int bits = held_bits;
            if (held) {
                each([&](uint32_t k, uint32_t i, uint64_t x) { all += !cut.keeps(k, i) ? 0 : counts ? 1 : x; });
                all = block_reduce(s, all);
                need = counts ? (uint64_t)top_k : by_k ? share(all) : row_share;
                if (need >= all) continue;
            } else {
                // 64 bins for one of the logits, or for a power of two of the weights
                const float rate = counts ? 64.0f : __builtin_fminf((float)(w.c * (64.0 / kPowers)), 1e30f);
                const auto bin_of = [&](float l) {
                    const float d = (finite_top - __builtin_fminf(l, __FLT_MAX__)) * rate;
                    return d < (float)(kSampleBins - 1) ? (int)d : kSampleBins - 1;
                };
                __syncthreads();
                for (int i = t; i < kSampleBins; i += kSampleThreads) s.bins[i] = 0;
                __syncthreads();
                for_row<T, 2>(row, a.vocab, [&](int i, T x) {
                    const uint32_t k = L::key(x);
                    if (k && cut.keeps(k, (uint32_t)i)) {
                        const uint64_t amount = counts ? 1 : w.of((float)x);
                        if (amount) add_to_bin(s, (uint32_t)bin_of((float)x), amount);
                    }
                });
                __syncthreads();
                for (int i = t; i < kSampleBins; i += kSampleThreads) all += s.bins[i];
                all = block_reduce(s, all);
                need = counts ? (uint64_t)top_k : share(all);
                if (need >= all) continue;
                find_bin<kSampleBins / 64>(s, need);
                const int bin = (int)s.bin;
                below = s.below;
                count = collect([&](uint32_t, T x) { return bin_of((float)x) == bin; });
                bits = L::BITS;
                if (count > kSampleList) {   // of equal or nearly equal ones: over the row again, by key and then by index
                    uint32_t key = 0;
                    uint64_t left = need;
#pragma unroll 1
                    for (int by_index = 0; by_index < 2; ++by_index) {
                        const uint32_t d = select(s, by_index ? index_bits : L::BITS, left, below, [&](auto&& f) {
                            for_row<T, 1>(row, a.vocab, [&](int i, T x) {
                                const uint32_t k = L::key(x);
                                if (k && cut.keeps(k, (uint32_t)i) && (!by_index || k == key))
                                    f(by_index ? (uint32_t)i : top_key - k, counts || by_index ? 1 : w.of((float)x));
                            });
                        });
                        if (by_index) {
                            cut = Cut{key, d};
                        } else {
                            key = top_key - d;
                            const uint64_t one = counts ? 1 : w.of(L::value(key));
                            left = (left - below + one - 1) / one;
                        }
                    }
                    continue;
                }
                load();
                need -= below;
            }
            // the key whose elements take the sum to `need`; of those, whose amounts are equal, the first ones
            const uint32_t key = top_key - select(s, bits, need, below, [&](auto&& f) {
                each([&](uint32_t k, uint32_t i, uint64_t x) {
                    if (cut.keeps(k, i)) f(top_key - k, counts ? 1 : x);
                });
            });
            const uint64_t one = counts ? 1 : w.of(L::value(key)), ties = (need - below + one - 1) / one;
            uint64_t equal = 0;
            each([&](uint32_t k, uint32_t i, uint64_t) { equal += k == key && cut.keeps(k, i); });
            uint32_t index = cut.key == key ? cut.index : 0xFFFFFFFFu;
            if (block_reduce(s, equal) > ties)
                index = select(s, index_bits, ties, below, [&](auto&& f) {
                    each([&](uint32_t k, uint32_t i, uint64_t) {
                        if (k == key && cut.keeps(k, i)) f(i, 1);
                    });
                });
            cut = Cut{key, index};
        }
        if (held) {
            uint64_t sum = 0;
            each([&](uint32_t k, uint32_t i, uint64_t& x) {
                x = cut.keeps(k, i) ? w.kept(L::value(k)) : 0;
                sum += x;
            });
            sum = block_reduce(s, sum);
            // the draw: indices in ascending order
            const uint64_t target = std::min<uint64_t>((uint64_t)((double)u * (double)sum), sum - 1);
            const uint32_t token = select(s, index_bits, target + 1, below, [&](auto&& f) {
                each([&](uint32_t, uint32_t i, uint64_t x) { f(i, x); });
            });
            each([&](uint32_t k, uint32_t i, uint64_t) {
                if (i == token) answer((int)token, w.log_of(L::value(k), temperature, sum));
            });
            return;
        }
        __syncthreads();
    }

    // the draw over the whole row: sums of tiles, then the tile that holds it
    const auto weight = [&](T l, int i) -> uint64_t {
        const uint32_t k = L::key(l);
        return k && cut.keeps(k, (uint32_t)i) ? w.kept((float)l) : 0;
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
        const Span at = span(tile);
        uint64_t sum = 0;
        if (at.n == L::VEC) {
            const typename L::vec v = *gptr<typename L::vec>(row + at.first);
#pragma unroll
            for (int e = 0; e < L::VEC; ++e) sum += weight(v[e], at.first + e);
        } else if (at.n) {
            sum = weight(row[at.first], at.first);
        }
        sum = prefix64(sum);
        if (lane == 63) s.tiles[tile] = sum;
    }
    __syncthreads();
    const int per = (tiles + kSampleThreads - 1) / kSampleThreads;
    uint64_t sum = 0, before;
    for (int i = t * per; i < std::min(tiles, (t + 1) * per); ++i) sum += s.tiles[i];
    const uint64_t total = block_reduce<Sum, true>(s, sum, &before);
    const uint64_t target = std::min<uint64_t>((uint64_t)((double)u * (double)total), total - 1);
    if (before <= target && target < before + sum) {
        for (int i = t * per; i < tiles; ++i) {
            if (target < before + s.tiles[i]) {
                s.bin = i;
                s.below = before;
                break;
            }
            before += s.tiles[i];
        }
    }
    __syncthreads();
    if (t >= 64) return;
    // its elements one by one: 64 neighbours at a time
    const Span at = span((int)s.bin);
    uint64_t lane_sum = 0;
#pragma unroll 1
    for (int e = 0; e < at.n; ++e) lane_sum += weight(row[at.first + e], at.first + e);
    uint64_t reached = s.below + prefix64(lane_sum) - lane_sum;
    if (reached <= target && target < reached + lane_sum) {
#pragma unroll 1
        for (int e = 0; e < at.n; ++e) {
            const int i = at.first + e;
            reached += weight(row[i], i);
            if (target < reached) {
                answer(i, w.log_of((float)row[i], temperature, total));
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
