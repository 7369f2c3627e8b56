// Rotary positions of libexq for gfx950 (exq_rotate): queries and keys of a
// block turned by their positions, in one launch.
//
// Pair i of a head, (u, v), at position p becomes
//   (u cos t - v sin t, u sin t + v cos t) * factor,   t = p * rate[i].
// Bound by the bytes of the heads in and out.  The angle is reduced to a part of
// a turn from its exact product, so far positions cost no accuracy; its sine
// and cosine then have the accuracy of 32 bits.  A thread has the
// same eight pairs of several heads of a row, so that the angles are paid for
// once.  4096 rows of 72 heads of 128 (151 MB in and out) take 26.3 to 29.3 us, 5.1
// to 5.7 TB/s, where a large copy has 5.3; one row takes 2.9 us on the GPU.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "exq_device_common.h"
#include "exq_internal.h"
#include "exq_operand.h"

namespace exq {

// Queries or keys: fp16 elements, strides in elements.
struct RotateHeads {
    const uint16_t* in;
    uint16_t* out;
    int64_t in_row, in_head, out_row, out_head;
};

struct RotateArgs {
    RotateHeads q, k;
    int q_heads, heads;       // heads: of both
    int rows, dim, part;
    int items;                // of a head: of PAIRS pairs each, then of the channels behind them (none in place)
    int turning;              // items of pairs
    int groups;               // threads that share a row's heads
    const double* rates;
    float factor;
    const int32_t* positions;
};

constexpr int kRotateThreads = 256;

// 1 / 2 pi in two numbers.  With the product of position and rate in two as well, what
// is left of a turn is good to 2^-50 for angles up to 2^40; rounding both to 64 bits
// leaves 2^-12.7 there and reaches 2^-20 at 2^32.  As fast: 29.3 us for 4096 rows of 72
// heads either way.
constexpr double kTurn = 0.15915494309189533577, kTurnRest = -9.839338337602413e-18;

// The PAIRS pairs of an item are channels a .. and b .. of the head (half
// layout), or 2 PAIRS neighbours (interleaved).
template <int PAIRS, bool INTERLEAVED>
__global__ __launch_bounds__(kRotateThreads) void rotate_kernel(RotateArgs a) {
    typedef _Float16 vec __attribute__((ext_vector_type(PAIRS)));
    const uint32_t id = blockIdx.x * (uint32_t)kRotateThreads + threadIdx.x;
    const uint32_t unit = id / (uint32_t)a.items, item = id - unit * (uint32_t)a.items;
    const uint32_t row = unit / (uint32_t)a.groups;
    if (row >= (uint32_t)a.rows) return;
    const int position = a.positions[row];
    if (position < 0) return;
    const bool turns = item < (uint32_t)a.turning;
    // the item's two runs of PAIRS channels
    int c0, c1;
    bool second = true;
    if (turns) {
        c0 = INTERLEAVED ? 2 * PAIRS * (int)item : PAIRS * (int)item;
        c1 = INTERLEAVED ? c0 + PAIRS : c0 + a.part / 2;
    } else {
        c0 = a.part + 2 * PAIRS * ((int)item - a.turning);
        c1 = c0 + PAIRS;
        second = c1 < a.dim;
    }
    float cs[PAIRS], sn[PAIRS];
    if (turns) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const double p = (double)position, rate = a.rates[PAIRS * item + i];
            const double t = p * rate, t_rest = __builtin_fma(p, rate, -t);
            const double turn = __builtin_fma(t, kTurn, -__builtin_rint(t * kTurn)) + __builtin_fma(t, kTurnRest, t_rest * kTurn);
            float s, c;
            sincospif(2.0f * (float)turn, &s, &c);
            cs[i] = c * a.factor;
            sn[i] = s * a.factor;
        }
    }
    for (int h = (int)(unit - row * (uint32_t)a.groups); h < a.heads; h += a.groups) {
        const bool is_q = h < a.q_heads;
        const RotateHeads& x = is_q ? a.q : a.k;
        const int64_t head = is_q ? h : h - a.q_heads;
        const uint16_t* in = x.in + row * x.in_row + head * x.in_head;
        uint16_t* out = x.out + row * x.out_row + head * x.out_head;
        vec u = *gptr<vec>(in + c0), v{};
        if (second) v = *gptr<vec>(in + c1);
        if (turns) {
            vec ru, rv;
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const float x0 = INTERLEAVED ? (2 * i < PAIRS ? u[2 * i % PAIRS] : v[2 * i % PAIRS]) : u[i];
                const float x1 = INTERLEAVED ? (2 * i + 1 < PAIRS ? u[(2 * i + 1) % PAIRS] : v[(2 * i + 1) % PAIRS]) : v[i];
                const _Float16 y0 = (_Float16)__builtin_fmaf(x0, cs[i], -(x1 * sn[i]));
                const _Float16 y1 = (_Float16)__builtin_fmaf(x0, sn[i], x1 * cs[i]);
                if (!INTERLEAVED) {
                    ru[i] = y0;
                    rv[i] = y1;
                } else {
                    if (2 * i < PAIRS) ru[2 * i % PAIRS] = y0;
                    else rv[2 * i % PAIRS] = y0;
                    if (2 * i + 1 < PAIRS) ru[(2 * i + 1) % PAIRS] = y1;
                    else rv[(2 * i + 1) % PAIRS] = y1;
                }
            }
            u = ru;
            v = rv;
        }
        *gptr_w<vec>(out + c0) = u;
        if (second) *gptr_w<vec>(out + c1) = v;
    }
}

}  // namespace exq

// =================================================================== host

using namespace exq;

extern "C" exq_status exq_rotate(const void* q, int64_t q_row_stride, int64_t q_head_stride, void* q_out,
                                 int64_t q_out_row_stride, int64_t q_out_head_stride, int q_heads, const void* k,
                                 int64_t k_row_stride, int64_t k_head_stride, void* k_out, int64_t k_out_row_stride,
                                 int64_t k_out_head_stride, int k_heads, int rows, int head_dim, int rotary_dim,
                                 int interleaved, const double* rates, float factor, const int32_t* positions,
                                 void* stream) {
    if (rows < 0 || q_heads < 0 || k_heads < 0 || q_heads > 65535 || k_heads > 65535 || q_heads + k_heads < 1)
        return fail(EXQ_ERR_INVALID_ARG, "rows=%d, heads %d and %d", rows, q_heads, k_heads);
    if (head_dim < 8 || head_dim % 8 || head_dim > 65536)
        return fail(EXQ_ERR_INVALID_ARG, "head_dim=%d is not a multiple of 8 in 8..65536", head_dim);
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim)
        return fail(EXQ_ERR_INVALID_ARG, "rotary_dim=%d is not even in 2..head_dim=%d", rotary_dim, head_dim);
    if (!__builtin_isfinite(factor)) return fail(EXQ_ERR_INVALID_ARG, "factor=%g", (double)factor);
    if (rows == 0) return EXQ_OK;
    if (!rates || !aligned(rates, 8)) return fail(EXQ_ERR_INVALID_ARG, "rates is NULL or misaligned");
    if (!positions || !aligned(positions, 4)) return fail(EXQ_ERR_INVALID_ARG, "positions is NULL or misaligned");
    const Operand in[2] = {{"q", q, q_row_stride, q_head_stride, rows, q_heads, head_dim},
                           {"k", k, k_row_stride, k_head_stride, rows, k_heads, head_dim}};
    const Operand out[2] = {{"q_out", q_out, q_out_row_stride, q_out_head_stride, rows, q_heads, head_dim},
                            {"k_out", k_out, k_out_row_stride, k_out_head_stride, rows, k_heads, head_dim}};
    exq_status st;
    bool in_place = true;
    for (int i = 0; i < 2; ++i) {
        if (!in[i].heads) continue;
        if ((st = check_operand(in[i])) != EXQ_OK || (st = check_operand(out[i])) != EXQ_OK) return st;
        if (!distinct(out[i])) return fail(EXQ_ERR_INVALID_ARG, "rows or heads of %s overlap themselves", out[i].name);
        if (ranges_meet(out[i].p, extent(out[i]), rates, 4 * (size_t)rotary_dim) ||
            ranges_meet(out[i].p, extent(out[i]), positions, 4 * (size_t)rows))
            return fail(EXQ_ERR_INVALID_ARG, "%s overlaps rates or positions", out[i].name);
        const bool same = in[i].p == out[i].p && (rows == 1 || in[i].row == out[i].row) && (in[i].heads == 1 || in[i].head == out[i].head);
        if (!same) {
            in_place = false;
            if (operands_meet(in[i], out[i]))
                return fail(EXQ_ERR_INVALID_ARG, "%s overlaps %s without being the same", out[i].name, in[i].name);
        }
    }
    if (q_heads && k_heads && (operands_meet(out[0], out[1]) || operands_meet(out[0], in[1]) || operands_meet(out[1], in[0])))
        return fail(EXQ_ERR_INVALID_ARG, "an output overlaps the other output or its input");
    // Eight pairs to a thread where vectors of 8 channels fit the pairs, else one, by single
    // channels: 4096 rows of 40 heads of 80 take 11.6 us where 32 channels turn, 24.7 where
    // 20 do and 23.5 where 40 do (in place 8.0, 9.7 and 14.3; a copy 8.2).
    const int pairs = rotary_dim % 16 == 0 ? 8 : 1;
    RotateArgs a;
    a.q = RotateHeads{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), q_row_stride, q_head_stride,
                      q_out_row_stride, q_out_head_stride};
    a.k = RotateHeads{static_cast<const uint16_t*>(k), static_cast<uint16_t*>(k_out), k_row_stride, k_head_stride,
                      k_out_row_stride, k_out_head_stride};
    a.q_heads = q_heads;
    a.heads = q_heads + k_heads;
    a.rows = rows;
    a.dim = head_dim;
    a.part = rotary_dim;
    a.turning = rotary_dim / (2 * pairs);
    a.items = a.turning + (in_place ? 0 : (head_dim - rotary_dim + 2 * pairs - 1) / (2 * pairs));
    a.groups = std::min(a.heads, 8);
    a.rates = rates;
    a.factor = factor;
    a.positions = positions;
    // few rows: a head to each thread
    while (a.groups < a.heads && (int64_t)rows * a.groups * a.items < 256 * 256) a.groups = std::min(a.heads, 2 * a.groups);
    const int64_t threads = (int64_t)rows * a.groups * a.items, blocks = (threads + kRotateThreads - 1) / kRotateThreads;
    if (blocks * kRotateThreads > kMaxLaunchThreads)
        return fail(EXQ_ERR_UNSUPPORTED, "%d rows of %d heads in one call", rows, a.heads);
    const dim3 grid((unsigned)blocks), block(kRotateThreads);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (pairs == 8) {
        if (interleaved) hipLaunchKernelGGL((rotate_kernel<8, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((rotate_kernel<8, false>), grid, block, 0, s, a);
    } else {
        if (interleaved) hipLaunchKernelGGL((rotate_kernel<1, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((rotate_kernel<1, false>), grid, block, 0, s, a);
    }
    return launched("rotate launch");
}
