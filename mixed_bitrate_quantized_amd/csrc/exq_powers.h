// Powers of two for the weights of exq_sample, in 64 bits.  Plain arithmetic, the same
// on the host.
#pragma once

#include <cstdint>

namespace exq {

constexpr int kPowers = 256;   // 2^(i / 256) in a table
constexpr double kLn2d = 0.69314718055994530942;

// 2^f for 0 <= f <= 1 from its series; the first term left out, ln(2)^16 / 16!, is
// below 2^-52 of it.
__host__ __device__ __forceinline__ double exp2_series(double f) {
    double p = 1.0;
#pragma unroll
    for (int i = 15; i >= 1; --i) p = __builtin_fma(p, f * (kLn2d / i), 1.0);
    return p;
}

// 2^(t / 256), t <= 0: an entry of the table (exp2_series(i / 256.0)) times 2^r, |r| <=
// 1/512, whose series is cut behind r^3: within 2^-45, the entry's error included.
__host__ __device__ __forceinline__ double power_of(const double* powers, double t) {
#pragma clang fp contract(off)   // the same bits wherever the compiler puts it
    constexpr double a = kLn2d / kPowers;
    t = __builtin_fmax(t, -256.0 * 1000);
    const double n = t + 6755399441055744.0;   // 1.5 * 2^52: rounds t, and leaves it in the sum's low bits
    const double f = t - (n - 6755399441055744.0);
    const int j = (int)(uint32_t)__builtin_bit_cast(uint64_t, n);
    const double near = powers[j & (kPowers - 1)];
    // |f| <= 1/2; the square's factor is a little above 1/2, which takes the error from 2^-42.7 to 2^-45.2
    const double q = __builtin_fma(f, __builtin_fma(f, a * a * a / 6, a * a * (0.5 + 0.0345178 * a * a / 4)), a);
    const double w = __builtin_fma(near * f, q, near);
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, w) + ((uint64_t)(uint32_t)((j >> 8) << 20) << 32));
}

}  // namespace exq
