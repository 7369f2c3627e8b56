// Low-rank adapters of many requests beside a shared projection (exq_lora_add)
// for gfx950:
//   out[r] = y[r] + s_a (x[r] A_a^T) B_a^T,   a = ids[r],
// for any mix of adapters in one call.
//
// Bound by the bytes of x, y, out and the adapters in use; for a few rows by
// the launches.  Three of them:
//   group   rows of one adapter are gathered into tiles, so that an adapter in
//           use is read once for a tile of its rows, in whatever order they come;
//   shrink  low = x A^T for a tile, K cut over waves and workgroups;
//   expand  out = y + s low B^T for a tile and a block of columns.
// Products run on v_mfma_f32_16x16x32_f16, sums are fp32.  low enters the second
// product as two fp16 numbers whose sum has 22 bits, scaled by a power of two
// to the row's largest: rounded to one fp16 it would cost half of the error
// the result's own rounding makes, and overflow beyond 65504.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>

#include "exq_device_common.h"
#include "exq_internal.h"
#include "exq_operand.h"

// Geometry of a stack of adapters and its borrowed weights (the
// exq_adapters_t handle).
struct exq_adapters {
    int count, K, N, rank;
    const uint16_t *a, *b;   // fp16 [count][rank][K], [count][N][rank]
    const float* scales;     // [count] or null
    const int32_t* ranks;    // [count] or null
};

namespace exq {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

// A tile: rows perm[start], .. perm[start + count - 1] of one adapter; adapter
// -1: rows without one, -2: rows whose number is out of range.
struct LoraTile {
    int32_t adapter, start, count, pad;
};

struct LoraArgs {
    const uint16_t *x, *y, *a, *b;
    uint16_t* out;
    int64_t x_row, y_row, out_row;
    int rows, K, N, rank, adapters;
    const float* scales;
    const int32_t *ranks, *ids;
    // workspace
    int32_t* tile_count;
    LoraTile* tiles;
    int32_t* perm;
    float* low;        // [splits][rows][rank]: parts of x A^T, rows in tiles' order
    int splits, slice;   // parts of K, and channels of one
    int columns;         // of an expanding workgroup
    bool in_place;
};

constexpr int kLoraGroupThreads = 1024;
constexpr int kLoraMaxAdapters = 8192;

// Counting sort of the rows by adapter.  Which of an adapter's rows share a tile
// depends on the order of atomics; a row's result does not depend on that.
__global__ __launch_bounds__(kLoraGroupThreads) void lora_group_kernel(LoraArgs a, int tile_rows) {
    __shared__ int32_t next[kLoraMaxAdapters + 2];
    __shared__ int32_t wave_rows[kLoraGroupThreads / 64], wave_tiles[kLoraGroupThreads / 64];
    const int t = threadIdx.x, lane = t % 64, wave = t / 64, bins = a.adapters + 2;
    for (int i = t; i < bins; i += kLoraGroupThreads) next[i] = 0;
    __syncthreads();
    const auto bin_of = [&](int id) { return id < 0 ? a.adapters : id < a.adapters ? id : a.adapters + 1; };
    for (int r = t; r < a.rows; r += kLoraGroupThreads) atomicAdd(&next[bin_of(a.ids[r])], 1);
    __syncthreads();
    int rows_before = 0, tiles_before = 0;
    for (int base = 0; base < bins; base += kLoraGroupThreads) {
        const int bin = base + t;
        const int n = bin < bins ? next[bin] : 0;
        // rows without an adapter need nothing where out is y
        const int tiles = bin == a.adapters && a.in_place ? 0 : (n + tile_rows - 1) / tile_rows;
        int rs = n, ts = tiles;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int u = __shfl_up(rs, d), v = __shfl_up(ts, d);
            if (lane >= d) rs += u, ts += v;
        }
        if (lane == 63) {
            wave_rows[wave] = rs;
            wave_tiles[wave] = ts;
        }
        __syncthreads();
        int row = rows_before + rs - n, tile = tiles_before + ts - tiles;
        for (int w = 0; w < kLoraGroupThreads / 64; ++w) {
            row += w < wave ? wave_rows[w] : 0;
            tile += w < wave ? wave_tiles[w] : 0;
            rows_before += wave_rows[w];
            tiles_before += wave_tiles[w];
        }
        if (bin < bins) {
            next[bin] = row;
            const int adapter = bin < a.adapters ? bin : bin == a.adapters ? -1 : -2;
            for (int i = 0; i < tiles; ++i)
                a.tiles[tile + i] = LoraTile{adapter, row + i * tile_rows, min(tile_rows, n - i * tile_rows), 0};
        }
        __syncthreads();
    }
    if (t == 0) *a.tile_count = tiles_before;
    for (int r = t; r < a.rows; r += kLoraGroupThreads) a.perm[atomicAdd(&next[bin_of(a.ids[r])], 1)] = r;
}

__device__ __forceinline__ h8 zero8() { return h8{}; }

constexpr int kShrinkWaves = 8;

// A wave's part of low^T = A x^T: 16 RT ranks by 16 TT rows.  Lane 16 q + i holds
// channels 8 q .. + 7 of rank i and of row i for each step of 32 channels, so
// both operands are loads of a row's neighbours.
template <int TT, int RT>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(LoraArgs a) {
    __shared__ f4 parts[kShrinkWaves / 2][RT * TT][64];
    const int tile_no = blockIdx.x / a.splits, split = blockIdx.x - tile_no * a.splits;
    if (tile_no >= *a.tile_count) return;
    const LoraTile tile = a.tiles[tile_no];
    if (tile.adapter < 0) return;
    const int t = threadIdx.x, wave = t / 64, lane = t % 64, i16 = lane % 16, q = lane / 16;
    const int rank0 = blockIdx.y * 16 * RT;
    const int rank = a.ranks ? min(max(a.ranks[tile.adapter], 0), a.rank) : a.rank;
    // the wave's channels
    const int per = a.slice / kShrinkWaves;
    const int k_begin = split * a.slice + wave * per, k_end = min(a.K, k_begin + per);
    const EXQ_GLOBAL uint16_t *xp[TT], *ap[RT];
    bool x_in[TT], a_in[RT];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        x_in[j] = 16 * j + i16 < tile.count;
        const int row = x_in[j] ? a.perm[tile.start + 16 * j + i16] : 0;
        xp[j] = gptr<uint16_t>(a.x + (int64_t)row * a.x_row);
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int r = rank0 + 16 * j + i16;
        a_in[j] = r < rank;
        ap[j] = gptr<uint16_t>(a.a + ((int64_t)tile.adapter * a.rank + (a_in[j] ? r : 0)) * a.K);
    }
    f4 acc[RT][TT];
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int m = 0; m < TT; ++m) acc[j][m] = f4{};
    constexpr int STEPS = TT + RT <= 4 ? 4 : 2;   // in flight
    for (int k0 = k_begin; k0 < k_end; k0 += 32 * STEPS) {
        h8 xs[STEPS][TT], as[STEPS][RT];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = k0 + 32 * s + 8 * q;
            const bool in = k < k_end;   // K and slices are multiples of 8
#pragma unroll
            for (int m = 0; m < TT; ++m) xs[s][m] = in && x_in[m] ? *(const EXQ_GLOBAL h8*)(xp[m] + k) : zero8();
#pragma unroll
            for (int j = 0; j < RT; ++j) as[s][j] = in && a_in[j] ? *(const EXQ_GLOBAL h8*)(ap[j] + k) : zero8();
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int m = 0; m < TT; ++m) acc[j][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(as[s][j], xs[s][m], acc[j][m], 0, 0, 0);
    }
    // the waves' sums, in a fixed order
#pragma unroll
    for (int half = kShrinkWaves / 2; half; half /= 2) {
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int m = 0; m < TT; ++m) parts[wave - half][j * TT + m][lane] = acc[j][m];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int m = 0; m < TT; ++m) acc[j][m] += parts[wave][j * TT + m][lane];
        __syncthreads();
    }
    if (wave) return;
    // lane 16 q + i: ranks 4 q .. + 3 of row i
#pragma unroll
    for (int m = 0; m < TT; ++m)
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int r = rank0 + 16 * j + 4 * q;
            if (x_in[m] && r < a.rank)   // a.rank is a multiple of 8
                *gptr_w<f4>(a.low + ((int64_t)split * a.rows + tile.start + 16 * m + i16) * a.rank + r) = acc[j][m];
        }
}

constexpr int kExpandWaves = 4;
constexpr int kLowPad = 8;   // fp16 after each row of low in LDS, against bank conflicts

// A wave takes 64 columns at a time: four products whose rows are columns 16 q +
// 4 m + i, so that a lane ends up with 16 neighbouring columns of one row.
template <int TT>
__global__ __launch_bounds__(64 * kExpandWaves) void lora_expand_kernel(LoraArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
    __shared__ float unscale[16 * TT];
    const int blocks = (a.N + a.columns - 1) / a.columns;
    const int tile_no = blockIdx.x / blocks, block = blockIdx.x - tile_no * blocks;
    if (tile_no >= *a.tile_count) return;
    const LoraTile tile = a.tiles[tile_no];
    const int t = threadIdx.x, lane = t % 64, wave = t / 64, i16 = lane % 16, q = lane / 16;
    const int n_begin = block * a.columns, n_end = min(a.N, n_begin + a.columns);
    if (tile.adapter < 0) {   // copied, or refused
        const uint16_t nan = 0x7E00;
        const h8 nans = {__builtin_bit_cast(_Float16, nan), __builtin_bit_cast(_Float16, nan), __builtin_bit_cast(_Float16, nan),
                         __builtin_bit_cast(_Float16, nan), __builtin_bit_cast(_Float16, nan), __builtin_bit_cast(_Float16, nan),
                         __builtin_bit_cast(_Float16, nan), __builtin_bit_cast(_Float16, nan)};
        for (int r = 0; r < tile.count; ++r) {
            const int64_t row = a.perm[tile.start + r];
            for (int n = n_begin + 8 * t; n < n_end; n += 8 * 64 * kExpandWaves)
                *gptr_w<h8>(a.out + row * a.out_row + n) = tile.adapter == -1 ? *gptr<h8>(a.y + row * a.y_row + n) : nans;
        }
        return;
    }
    const int rank = a.ranks ? min(max(a.ranks[tile.adapter], 0), a.rank) : a.rank;
    const int padded = (a.rank + 31) / 32 * 32, pitch = padded + kLowPad;
    uint16_t *hi = lds, *lo = lds + 16 * TT * pitch;
    const float scale = a.scales ? a.scales[tile.adapter] : 1.0f;
    // low: four lanes a row add up its parts, find its largest and cut it in two
    {
        constexpr int LANES = 64 * kExpandWaves / (16 * TT);   // of a row: 16 or 4
        const int r = t / LANES, first = t % LANES;
        const float* from = a.low + (int64_t)(tile.start + r) * a.rank;
        const auto value = [&](int j) {
            float v = 0.0f;
            if (r < tile.count && j < rank)
                for (int s = 0; s < a.splits; ++s) v += from[(int64_t)s * a.rows * a.rank + j];
            return v;
        };
        float most = 0.0f;
        for (int j = first; j < rank; j += LANES) {
            const float v = __builtin_fabsf(value(j));
            most = v < __builtin_huge_valf() ? __builtin_fmaxf(most, v) : most;
        }
#pragma unroll
        for (int d = 1; d < LANES; d *= 2) most = __builtin_fmaxf(most, __shfl_xor(most, d));
        // |low| * 2^e below 2^15
        int e = 0;
        if (most > 0.0f) e = 15 - (__builtin_amdgcn_frexp_expf(most));
        e = min(e, 126);
        for (int j = first; j < padded; j += LANES) {
            const float v = __builtin_ldexpf(value(j), e);
            const _Float16 h = (_Float16)v;
            hi[r * pitch + j] = __builtin_bit_cast(uint16_t, h);
            lo[r * pitch + j] = f32_to_f16_bits(v - (float)h);
        }
        if (first == 0) unscale[r] = __builtin_ldexpf(scale, -e);
    }
    __syncthreads();
    int64_t row[TT];
    bool in[TT];
    float f[TT];
#pragma unroll
    for (int m = 0; m < TT; ++m) {
        in[m] = 16 * m + i16 < tile.count;
        row[m] = in[m] ? a.perm[tile.start + 16 * m + i16] : 0;
        f[m] = unscale[16 * m + i16];
    }
    const uint16_t* b = a.b + (int64_t)tile.adapter * a.N * a.rank;
    for (int n0 = n_begin + 64 * wave; n0 < n_end; n0 += 64 * kExpandWaves) {
        f4 acc[4][TT];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < TT; ++j) acc[m][j] = f4{};
        for (int k = 0; k < rank; k += 32) {
            h8 bs[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int n = n0 + 16 * (i16 / 4) + 4 * m + i16 % 4, j = k + 8 * q;
                h8 v = n < n_end && j < rank ? *gptr<h8>(b + (int64_t)n * a.rank + j) : zero8();
                if (j + 8 > rank)   // what lies behind the adapter's own rank may be anything
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = j + e < rank ? v[e] : (_Float16)0.0f;
                bs[m] = v;
            }
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                const h8 h = *reinterpret_cast<const h8*>(hi + (16 * j + i16) * pitch + k + 8 * q);
                const h8 l = *reinterpret_cast<const h8*>(lo + (16 * j + i16) * pitch + k + 8 * q);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(bs[m], h, acc[m][j], 0, 0, 0);
                    acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(bs[m], l, acc[m][j], 0, 0, 0);
                }
            }
        }
        const int n = n0 + 16 * q;
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            if (!in[j]) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (n + 8 * half >= n_end) continue;   // N and blocks are multiples of 8
                h8 v = *gptr<h8>(a.y + row[j] * a.y_row + n + 8 * half);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = (_Float16)__builtin_fmaf(acc[2 * half + e / 4][j][e % 4], f[j], (float)v[e]);
                *gptr_w<h8>(a.out + row[j] * a.out_row + n + 8 * half) = v;
            }
        }
    }
}

}  // namespace exq

// =================================================================== host

using namespace exq;

namespace {

// Shape of a call.
struct LoraPlan {
    int tile_rows, tiles, splits, slice;
    size_t tiles_at, perm_at, low_at, bytes;   // of the workspace
};

exq_status plan_lora(const exq_adapters* h, int rows, LoraPlan* p) {
    if (!h) return fail(EXQ_ERR_INVALID_ARG, "adapters is NULL");
    if (rows < 0) return fail(EXQ_ERR_INVALID_ARG, "rows=%d", rows);
    p->tile_rows = rows >= 512 && h->rank <= 128 ? 64 : 16;
    p->tiles = (int)std::min<int64_t>(rows, (int64_t)rows / p->tile_rows + h->count + 2);
    // a wave has 128 channels at least; about 512 workgroups
    const int rank_blocks = (h->rank + 31) / 32;
    const int most = std::max(1, (h->K + 128 * kShrinkWaves - 1) / (128 * kShrinkWaves));
    const int busy = std::max(1, std::min(p->tiles, rows / p->tile_rows + 1)) * rank_blocks;
    p->splits = std::max(1, std::min(most, 512 / busy));
    const int unit = 32 * kShrinkWaves;
    p->slice = ((h->K + p->splits - 1) / p->splits + unit - 1) / unit * unit;
    p->splits = (h->K + p->slice - 1) / p->slice;
    p->tiles_at = 16;
    p->perm_at = p->tiles_at + sizeof(LoraTile) * (size_t)p->tiles;
    p->low_at = (p->perm_at + 4 * (size_t)rows + 15) / 16 * 16;
    p->bytes = rows ? p->low_at + 4 * (size_t)p->splits * rows * h->rank : 0;
    return EXQ_OK;
}

}  // namespace

extern "C" {

exq_status exq_adapters_create(int count, int K, int N, int rank, const void* a, const void* b, const float* scales,
                               const int32_t* ranks, exq_adapters_t* out) {
    if (!out) return fail(EXQ_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (count < 1 || K < 8 || N < 8 || rank < 8 || K % 8 || N % 8 || rank % 8)
        return fail(EXQ_ERR_INVALID_ARG, "count=%d K=%d N=%d rank=%d: K, N and rank must be positive multiples of 8", count, K, N, rank);
    if (count > kLoraMaxAdapters) return fail(EXQ_ERR_UNSUPPORTED, "%d adapters: over %d", count, kLoraMaxAdapters);
    if (rank > 256) return fail(EXQ_ERR_UNSUPPORTED, "rank=%d over 256", rank);
    if (K > 1 << 20 || N > 1 << 20) return fail(EXQ_ERR_UNSUPPORTED, "K=%d N=%d over 2^20", K, N);
    if (!a || !b || !aligned(a, 16) || !aligned(b, 16)) return fail(EXQ_ERR_INVALID_ARG, "a or b is NULL or not 16-byte aligned");
    if (!aligned(scales, 4) || !aligned(ranks, 4)) return fail(EXQ_ERR_INVALID_ARG, "scales or ranks is misaligned");
    exq_adapters* h = new (std::nothrow) exq_adapters();
    if (!h) return fail(EXQ_ERR_OOM, "host allocation");
    *h = exq_adapters{count, K, N, rank, static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b), scales, ranks};
    *out = h;
    return EXQ_OK;
}

void exq_adapters_destroy(exq_adapters_t h) { delete h; }

size_t exq_lora_workspace_bytes(exq_adapters_t h, int rows) {
    LoraPlan p;
    return plan_lora(h, rows, &p) == EXQ_OK ? p.bytes : 0;
}

exq_status exq_lora_add(exq_adapters_t h, const void* x, int64_t x_row_stride, int rows, const int32_t* ids, const void* y,
                        int64_t y_row_stride, void* out, int64_t out_row_stride, void* workspace, size_t workspace_bytes,
                        void* stream) {
    LoraPlan p;
    exq_status st = plan_lora(h, rows, &p);
    if (st != EXQ_OK || rows == 0) return st;
    const Operand xo{"x", x, x_row_stride, 0, rows, 1, h->K}, yo{"y", y, y_row_stride, 0, rows, 1, h->N},
        oo{"out", out, out_row_stride, 0, rows, 1, h->N};
    if ((st = check_operand(xo)) != EXQ_OK || (st = check_operand(yo)) != EXQ_OK || (st = check_operand(oo)) != EXQ_OK) return st;
    if (!ids || !aligned(ids, 4)) return fail(EXQ_ERR_INVALID_ARG, "ids is NULL or misaligned");
    if (!distinct(oo)) return fail(EXQ_ERR_INVALID_ARG, "rows of out overlap themselves");
    const bool in_place = y == out && (rows == 1 || y_row_stride == out_row_stride);
    if (operands_meet(xo, oo) || (!in_place && operands_meet(yo, oo)))
        return fail(EXQ_ERR_INVALID_ARG, "out overlaps x, or y without being the same");
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < p.bytes)
        return fail(EXQ_ERR_INVALID_ARG, "workspace of %zu bytes: %zu 16-byte aligned ones are needed", workspace_bytes, p.bytes);
    const struct {
        const char* name;
        const void* p;
        size_t bytes;
    } read[] = {{"ids", ids, 4 * (size_t)rows},
                {"a", h->a, 2 * (size_t)h->count * h->rank * h->K},
                {"b", h->b, 2 * (size_t)h->count * h->N * h->rank},
                {"scales", h->scales, h->scales ? 4 * (size_t)h->count : 0},
                {"ranks", h->ranks, h->ranks ? 4 * (size_t)h->count : 0}};
    for (const auto& z : read)
        if (z.bytes && (ranges_meet(out, extent(oo), z.p, z.bytes) || ranges_meet(workspace, p.bytes, z.p, z.bytes)))
            return fail(EXQ_ERR_INVALID_ARG, "out or the workspace overlaps %s", z.name);
    if (ranges_meet(workspace, p.bytes, x, extent(xo)) || ranges_meet(workspace, p.bytes, y, extent(yo)) ||
        ranges_meet(workspace, p.bytes, out, extent(oo)))
        return fail(EXQ_ERR_INVALID_ARG, "workspace overlaps x, y or out");
    char* ws = static_cast<char*>(workspace);
    LoraArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.y = static_cast<const uint16_t*>(y);
    a.a = h->a;
    a.b = h->b;
    a.out = static_cast<uint16_t*>(out);
    a.x_row = x_row_stride;
    a.y_row = y_row_stride;
    a.out_row = out_row_stride;
    a.rows = rows;
    a.K = h->K;
    a.N = h->N;
    a.rank = h->rank;
    a.adapters = h->count;
    a.scales = h->scales;
    a.ranks = h->ranks;
    a.ids = ids;
    a.tile_count = reinterpret_cast<int32_t*>(ws);
    a.tiles = reinterpret_cast<LoraTile*>(ws + p.tiles_at);
    a.perm = reinterpret_cast<int32_t*>(ws + p.perm_at);
    a.low = reinterpret_cast<float*>(ws + p.low_at);
    a.splits = p.splits;
    a.slice = p.slice;
    a.in_place = in_place;
    // a wave's 64 columns at a time, blocks that make about 1024 workgroups
    const int unit = 64 * kExpandWaves, units = (h->N + unit - 1) / unit;
    const int busy = std::min(p.tiles, rows / p.tile_rows + 1);
    a.columns = unit * std::max<int>(1, (int)std::min<int64_t>(units, (int64_t)units * busy / 1024));
    const int blocks = (h->N + a.columns - 1) / a.columns, rank_blocks = (h->rank + 31) / 32;
    if ((int64_t)p.tiles * std::max(blocks, p.splits * rank_blocks) > kMaxLaunchThreads / 1024)
        return fail(EXQ_ERR_UNSUPPORTED, "%d rows in one call", rows);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(lora_group_kernel, dim3(1), dim3(kLoraGroupThreads), 0, s, a, p.tile_rows);
    if ((st = launched("adapters group launch")) != EXQ_OK) return st;
    const dim3 shrink_grid((unsigned)(p.tiles * p.splits), (unsigned)rank_blocks), shrink_block(64 * kShrinkWaves);
    const dim3 expand_grid((unsigned)(p.tiles * blocks)), expand_block(64 * kExpandWaves);
    const int pitch = (h->rank + 31) / 32 * 32 + kLowPad;
    const unsigned lds = 2u * 2u * p.tile_rows * pitch;
    if (p.tile_rows == 64) {
        hipLaunchKernelGGL((lora_shrink_kernel<4, 2>), shrink_grid, shrink_block, 0, s, a);
        if ((st = launched("adapters shrink launch")) != EXQ_OK) return st;
        hipLaunchKernelGGL((lora_expand_kernel<4>), expand_grid, expand_block, lds, s, a);
    } else {
        hipLaunchKernelGGL((lora_shrink_kernel<1, 2>), shrink_grid, shrink_block, 0, s, a);
        if ((st = launched("adapters shrink launch")) != EXQ_OK) return st;
        hipLaunchKernelGGL((lora_expand_kernel<1>), expand_grid, expand_block, lds, s, a);
    }
    return launched("adapters expand launch");
}

}  // extern "C"
