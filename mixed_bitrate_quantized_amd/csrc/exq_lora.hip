// Low-rank adapters of many requests beside a shared projection (exq_lora_add)
// for gfx950:
//   out[r] = y[r] + s_a (x[r] A_a^T) B_a^T,   a = ids[r],
// for any mix of adapters in one call.
//
// Bound by the bytes of x, y, out and the adapters in use; for a few rows by
// the launches.  Rows of one adapter are gathered into tiles, so that an adapter
// in use is read once for a tile of its rows, in whatever order they come:
//   group   the rows sorted by adapter: up to 64 rows by every wave for itself, up to
//           4096 by every shrinking workgroup, more by a launch of their own;
//   shrink  low = x A^T for 16 or 32 rows, K cut over waves and workgroups;
//   expand  out = y + s low B^T for a tile and a block of columns.
// A few rows of small adapters take one launch, which does all of that.
// 48 rows of 16 adapters of rank 64 beside 8192 x 28672 take 23.3 us: shrinking 7,
// expanding 15 of them, B's lines (59 MB) at 3.9 TB/s with the start.  2048 rows of 6
// adapters of rank 32 beside 8192 x 8192 take 41.0: 105 MB; shrinking 18.4 (grouping
// 3 of them), expanding 18, 67 MB at 3.7 TB/s.
// Products run on v_mfma_f32_16x16x32_f16, sums are fp32.  low enters the second
// product as two fp16 numbers whose sum has 22 bits, scaled by a power of two
// to the row's largest: rounded to one fp16 it would cost half of the error
// the result's own rounding makes, and overflow beyond 65504.  Rows with a rank
// too far below the largest for fp16's range take the second product in fp32.
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

// A tile: up to 16 or 64 rows of one adapter, its rank and scale; adapter -1:
// rows without one, -2: rows whose number is out of range.  count 0: none.
struct LoraTile {
    int32_t adapter, count, rank;
    float scale;
};

struct LoraArgs {
    const uint16_t *x, *y, *a, *b;
    uint16_t* out;
    int64_t x_row, y_row, out_row;
    int rows, K, N, rank, adapters;
    const float* scales;
    const int32_t *ranks, *ids;
    // workspace
    LoraTile* tiles;
    int32_t* tile_rows;   // of each tile
    int32_t* place;       // of each row among its adapter's
    float* low;           // [splits][rows][rank]: parts of x A^T
    int splits, slice;   // parts of K, and channels of one
    int blocks, columns;   // expanding workgroups of a tile, and columns of one
    bool in_place;
};

constexpr int kLoraFew = 64;     // rows that a wave groups by itself
constexpr int kLoraSplits = 8;   // parts of K at most

__device__ __forceinline__ int lora_rank(const LoraArgs& a, int adapter) {
    return adapter < 0 ? 0 : a.ranks ? min(max(a.ranks[adapter], 0), a.rank) : a.rank;
}
__device__ __forceinline__ float lora_scale(const LoraArgs& a, int adapter) {
    return a.scales && adapter >= 0 ? a.scales[adapter] : 1.0f;
}

// Tile `no` of tiles of T rows, lane i with the row of slot i.
template <int T> __device__ __forceinline__ LoraTile lora_tile(const LoraArgs& a, int no, int& row) {
    const int lane = threadIdx.x & 63;
    const LoraTile tile = a.tiles[no];
    row = a.tile_rows[(int64_t)no * T + lane % T];
    if (lane >= tile.count) row = 0;
    return tile;
}

// The same for up to 64 rows without the table: every wave groups them for
// itself, an adapter at a time, in order of its first row.
template <int T> __device__ __forceinline__ LoraTile lora_tile_of_few(const LoraArgs& a, int no, int& row) {
    const int lane = threadIdx.x & 63;
    int id = lane < a.rows ? a.ids[lane] : -1;
    id = id < 0 ? -1 : id < a.adapters ? id : -2;
    // rows without an adapter need nothing where out is y
    uint64_t left = __ballot(lane < a.rows && !(a.in_place && id == -1));
    row = 0;
    while (left) {
        const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t same = __ballot(id == one) & left;
        const int n = __builtin_popcountll(same), tiles = (n + T - 1) / T;
        if (no < tiles) {
            // the place of the bit that is the lane's in `same`
            int nth = no * T + lane;
#pragma unroll
            for (int w = 32; w; w /= 2) {
                const int below = __builtin_popcountll(same >> row & ((1ull << w) - 1));
                if (nth >= below) {
                    nth -= below;
                    row += w;
                }
            }
            const int count = min(T, n - no * T);
            if (lane >= count) row = 0;
            return LoraTile{one, count, lora_rank(a, one), lora_scale(a, one)};
        }
        no -= tiles;
        left &= ~same;
    }
    return LoraTile{-1, 0, 0, 0.0f};
}

// The same for up to kLoraSome rows by a workgroup of THREADS, which counts the rows
// of all adapters (THREADS - 2 at most), finds the tile's and then its rows among
// theirs, in order of the threads that hold them.
constexpr int kLoraSome = 4096;
template <int T, int THREADS> __device__ __forceinline__ LoraTile lora_tile_of_some(const LoraArgs& a, int no, int& row) {
    constexpr int EACH = kLoraSome / THREADS, WAVES = THREADS / 64;
    static_assert(WAVES == 8 || WAVES == 16, "a row of lanes adds up the waves");
    __shared__ int32_t bin_rows[THREADS], tile_rows[T], found[3];
    __shared__ uint64_t waves[2][16];
    const int t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
    const auto before_of = [&](uint64_t (&sums)[16], int x) {   // the threads' before; a barrier is in it
        const uint64_t upto = prefix64((uint64_t)x);
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        const uint64_t to = prefix16(sums[lane & 15]);
        return (int)(upto - x + (wave ? lane_value(to, wave - 1) : 0));
    };
    int bin[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const int r = t + e * THREADS, i = r < a.rows ? a.ids[r] : -1;
        bin[e] = r >= a.rows ? -1 : i < 0 ? a.adapters : i < a.adapters ? i : a.adapters + 1;
    }
    bin_rows[t] = 0;
    if (t < 32) waves[t / 16][t % 16] = 0;
    if (t == 0) found[2] = 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        // those of the first lane's adapter at once: rows often come in runs
        const int one = __builtin_amdgcn_readfirstlane(bin[e]);
        const uint64_t same = __ballot(bin[e] == one);
        if (one >= 0 && lane == 0) atomicAdd(&bin_rows[one], __builtin_popcountll(same));
        if (bin[e] >= 0 && bin[e] != one) atomicAdd(&bin_rows[bin[e]], 1);
    }
    __syncthreads();
    const int mine = bin_rows[t];
    // rows without an adapter need nothing where out is y
    const int tiles = t == a.adapters && a.in_place ? 0 : (mine + T - 1) / T, first = before_of(waves[0], tiles);
    if (first <= no && no < first + tiles) {
        found[0] = t;
        found[1] = (no - first) * T;
        found[2] = mine;
    }
    __syncthreads();
    row = 0;
    if (found[2] == 0) return LoraTile{-1, 0, 0, 0.0f};
    const int its = found[0], from = found[1], adapter = its < a.adapters ? its : its == a.adapters ? -1 : -2;
    const int count = min(T, found[2] - from), rank = lora_rank(a, adapter);
    const float scale = lora_scale(a, adapter);
    int same = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) same += bin[e] == its;
    int place = before_of(waves[1], same) - from;
#pragma unroll
    for (int e = 0; e < EACH; ++e)
        if (bin[e] == its) {
            if (place >= 0 && place < T) tile_rows[place] = t + e * THREADS;
            ++place;
        }
    __syncthreads();
    if (lane < count) row = tile_rows[lane % T];
    return LoraTile{adapter, count, rank, scale};
}

constexpr int kLoraGroupThreads = 1024;
constexpr int kLoraGroupEach = 8;   // rows whose places a thread keeps in registers
constexpr int kLoraMaxAdapters = 8192;

// Counting sort of more rows by adapter.  Which of an adapter's rows share a tile
// depends on the order of atomics; a row's result does not depend on that.
// One workgroup, a chain of look-ups: 2048 rows of 6 adapters would take 5.8 us,
// the shrinking workgroups' own look 3.
__global__ __launch_bounds__(kLoraGroupThreads) void lora_group_kernel(LoraArgs a, int T, int most_tiles) {
    __shared__ int32_t bin_rows[kLoraMaxAdapters + 2], first_tile[kLoraMaxAdapters + 2];
    __shared__ int32_t wave_tiles[kLoraGroupThreads / 64];
    const int t = threadIdx.x, lane = t % 64, wave = t / 64, bins = a.adapters + 2;
    int id[kLoraGroupEach], place[kLoraGroupEach];
    const auto bin_of = [&](int i) { return i < 0 ? a.adapters : i < a.adapters ? i : a.adapters + 1; };
#pragma unroll
    for (int i = 0; i < kLoraGroupEach; ++i) id[i] = t + i * kLoraGroupThreads < a.rows ? a.ids[t + i * kLoraGroupThreads] : 0;
    for (int i = t; i < bins; i += kLoraGroupThreads) bin_rows[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kLoraGroupEach; ++i)
        if (t + i * kLoraGroupThreads < a.rows) place[i] = atomicAdd(&bin_rows[bin_of(id[i])], 1);
    for (int r = t + kLoraGroupEach * kLoraGroupThreads; r < a.rows; r += kLoraGroupThreads)
        a.place[r] = atomicAdd(&bin_rows[bin_of(a.ids[r])], 1);
    __syncthreads();
    int tiles_before = 0;
    for (int base = 0; base < bins; base += kLoraGroupThreads) {
        const int bin = base + t, adapter = bin < a.adapters ? bin : bin == a.adapters ? -1 : -2;
        const int n = bin < bins ? bin_rows[bin] : 0;
        // rows without an adapter need nothing where out is y
        const int tiles = adapter == -1 && a.in_place ? 0 : (n + T - 1) / T;
        const int rank = n ? lora_rank(a, adapter) : 0;
        const float scale = n ? lora_scale(a, adapter) : 0.0f;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int u = __shfl_up(sum, d);
            if (lane >= d) sum += u;
        }
        if (lane == 63) wave_tiles[wave] = sum;
        __syncthreads();
        int tile = tiles_before + sum - tiles;
        for (int w = 0; w < kLoraGroupThreads / 64; ++w) {
            tile += w < wave ? wave_tiles[w] : 0;
            tiles_before += wave_tiles[w];
        }
        if (bin < bins) {
            first_tile[bin] = tiles ? tile : -1;
            for (int i = 0; i < tiles; ++i) a.tiles[tile + i] = LoraTile{adapter, min(T, n - i * T), rank, scale};
        }
        __syncthreads();
    }
    for (int i = tiles_before + t; i < most_tiles; i += kLoraGroupThreads) a.tiles[i] = LoraTile{-1, 0, 0, 0.0f};
    const auto put = [&](int r, int i, int at) {
        const int first = first_tile[bin_of(i)];
        if (first >= 0) a.tile_rows[(int64_t)first * T + at] = r;
    };
#pragma unroll
    for (int i = 0; i < kLoraGroupEach; ++i)
        if (t + i * kLoraGroupThreads < a.rows) put(t + i * kLoraGroupThreads, id[i], place[i]);
    for (int r = t + kLoraGroupEach * kLoraGroupThreads; r < a.rows; r += kLoraGroupThreads) put(r, a.ids[r], a.place[r]);
}

// A wave's part of low^T = A x^T: 16 RT ranks by 16 TT rows (of a tile of T), K
// cut over W waves.  Lane 16 q + i holds channels 8 q .. + 7 of rank i and of row i
// for each step of 32 channels, so both operands are loads of a row's neighbours.
// All of a wave's STEPS steps are in flight at once where K is cut that fine.
// Tiles of 64 rows are shrunk 32 at a time, to read A half as often: x from
// memory and A from L2 add up (2048 rows of 8192 at rank 32 took 21 us by 16,
// 12 of them without A, 13 without x).
constexpr int shrink_waves(int T) { return T == 64 ? 16 : 8; }
constexpr int shrink_rows(int T) { return T == 64 ? 2 : 1; }   // in units of 16
template <int TT, int RT> constexpr int kShrinkSteps = RT == 4 && TT == 2 ? 2 : 4;

// By whom a tile's rows are looked for.
enum LoraGroup { kByWave, kByWorkgroup, kByLaunch };

template <LoraGroup GROUP, int T, int RT>
__global__ __launch_bounds__(64 * shrink_waves(T)) void lora_shrink_kernel(LoraArgs a) {
    constexpr int TT = shrink_rows(T), W = shrink_waves(T);
    __shared__ f4 parts[W / 2][RT * TT][64];
    constexpr int SUBS = T / (16 * TT);
    const int split = blockIdx.x % a.splits, no = blockIdx.x / a.splits / SUBS, slot0 = blockIdx.x / a.splits % SUBS * 16 * TT;
    const int t = threadIdx.x, wave = t / 64, lane = t % 64, i16 = lane % 16, q = lane / 16;
    int rows_of_tile;
    LoraTile tile;
    if constexpr (GROUP == kByWave) tile = lora_tile_of_few<T>(a, no, rows_of_tile);
    else if constexpr (GROUP == kByWorkgroup) tile = lora_tile_of_some<T, 64 * W>(a, no, rows_of_tile);
    else tile = lora_tile<T>(a, no, rows_of_tile);
    if (GROUP != kByLaunch && split == 0 && slot0 == 0 && blockIdx.y == 0 && wave == 0) {   // for lora_expand_kernel
        if (lane == 0) a.tiles[no] = tile;
        if (lane < T) a.tile_rows[no * T + lane] = rows_of_tile;
    }
    if (tile.adapter < 0 || slot0 >= tile.count) return;
    const int rank0 = blockIdx.y * 16 * RT;
    // the wave's channels
    const int per = a.slice / W;
    const int k_begin = split * a.slice + wave * per, k_end = min(a.K, k_begin + per);
    const EXQ_GLOBAL uint16_t *xp[TT], *ap[RT];
    int row[TT];
    bool x_in[TT], a_in[RT];
#pragma unroll
    for (int m = 0; m < TT; ++m) {
        x_in[m] = slot0 + 16 * m + i16 < tile.count;
        row[m] = __shfl(rows_of_tile, slot0 + 16 * m + i16);
        xp[m] = gptr<uint16_t>(a.x + (int64_t)row[m] * a.x_row);
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int r = rank0 + 16 * j + i16;
        a_in[j] = r < tile.rank;
        ap[j] = gptr<uint16_t>(a.a + ((int64_t)tile.adapter * a.rank + (a_in[j] ? r : 0)) * a.K);
    }
    f4 acc[RT][TT];
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int m = 0; m < TT; ++m) acc[j][m] = f4{};
    constexpr int STEPS = kShrinkSteps<TT, RT>;
    for (int k0 = k_begin; k0 < k_end; k0 += 32 * STEPS) {
        h8 xs[STEPS][TT], as[STEPS][RT];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = k0 + 32 * s + 8 * q;
            const bool in = k < k_end;   // K and slices are multiples of 8
#pragma unroll
            for (int m = 0; m < TT; ++m) xs[s][m] = in && x_in[m] ? *(const EXQ_GLOBAL h8*)(xp[m] + k) : h8{};
#pragma unroll
            for (int j = 0; j < RT; ++j) as[s][j] = in && a_in[j] ? *(const EXQ_GLOBAL h8*)(ap[j] + k) : h8{};
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
    for (int half = W / 2; half; half /= 2) {
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
                *gptr_w<f4>(a.low + ((int64_t)split * a.rows + row[m]) * a.rank + r) = acc[j][m];
        }
}

// Rows without an adapter are copied, those of a number out of range refused.
__device__ __forceinline__ void lora_copy(const LoraArgs& a, const LoraTile& tile, int rows_of_tile, int n_begin, int n_end) {
    const _Float16 nan = __builtin_bit_cast(_Float16, (uint16_t)0x7E00);
    const h8 nans = {nan, nan, nan, nan, nan, nan, nan, nan};
    // Runs of 8 columns of all rows dealt out over the threads, four of each under way
    // (1074 rows of 8192 x 8192, 97 of them without an adapter: 25.9 us, row by row 43).
    const int runs = (n_end - n_begin) / 8, all = tile.count * runs;
    for (int i0 = 0; i0 < all; i0 += 4 * (int)blockDim.x) {
        h8 x[4];
        int64_t row[4];
        int n[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int i = i0 + m * (int)blockDim.x + (int)threadIdx.x, r = min(i / runs, tile.count - 1);
            row[m] = __shfl(rows_of_tile, r);
            n[m] = i < all ? n_begin + 8 * (i - r * runs) : -1;
            x[m] = tile.adapter == -1 && n[m] >= 0 ? *gptr<h8>(a.y + row[m] * a.y_row + n[m]) : nans;
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
            if (n[m] >= 0) *gptr_w<h8>(a.out + row[m] * a.out_row + n[m]) = x[m];
    }
}

// Power of two that takes a row's largest finite |low| below 2^15, and the cut of a value in two.
__device__ __forceinline__ int lora_shift(float most) { return most > 0.0f ? min(15 - __builtin_amdgcn_frexp_expf(most), 126) : 0; }
__device__ __forceinline__ void lora_cut(float x, int e2, _Float16& high, _Float16& rest) {
    x = __builtin_ldexpf(x, e2);
    high = (_Float16)x;
    rest = (_Float16)(x - (float)high);
}
// What takes a sum back: the adapter's scale over the row's.  Past fp32's range it stays
// at the largest: what it meets is 0, or far beyond fp16 either way.
__device__ __forceinline__ float lora_unscale(float scale, int e2) {
    const float f = __builtin_ldexpf(scale, -e2);
    return __builtin_fabsf(scale) <= __FLT_MAX__ ? __builtin_fmaxf(__builtin_fminf(f, __FLT_MAX__), -__FLT_MAX__) : f;
}
// Whether the cut loses more than 2^-18 of the value.  The rest is good to 2^-22 of it
// or, subnormal, to 2^-25, so values from 2^-7 on lose less; they are 2^21 below the
// largest.  (2^-18 of each rank's product is half of the 64 * 2^-23 that the stated
// accuracy has beside the sums.  Of a million normally distributed ranks about one is
// as small.)
__device__ __forceinline__ bool lora_lost(float x, int e2) {
    x = __builtin_fabsf(__builtin_ldexpf(x, e2));
    return x > 0.0f && x < 0x1p-7f;
}

// The second product of one row in fp32, its products `low` of the first in LDS
// (16-byte aligned, to a multiple of 8), of columns `first` and on, `step` apart.  By
// the row's own values alone, as in the tiles: what shares a tile with it does not
// change it.  48 rows of rank 64 beside 8192 x 28672 take 23.2 us, with one such row
// 26.4, with nothing else 66; 2048 rows of rank 32 beside 8192 x 8192 38, 38 and 205;
// one row of rank 16 8.8 and 9.2.
__device__ __forceinline__ void lora_expand_row(const LoraArgs& a, const LoraTile& tile, int64_t row, int first, int n_end, int step, const float* low) {
    const uint16_t* b = a.b + (int64_t)tile.adapter * a.N * a.rank;
    for (int c = first; c < n_end; c += step) {
        float sum = 0.0f;
#pragma unroll 4
        for (int j = 0; j < tile.rank; j += 8) {   // a.rank is a multiple of 8
            const h8 x = *gptr<h8>(b + (int64_t)c * a.rank + j);
            const f4 l[2] = {*reinterpret_cast<const f4*>(low + j), *reinterpret_cast<const f4*>(low + j + 4)};
#pragma unroll
            for (int e = 0; e < 8; ++e)   // what lies behind the adapter's own rank may be anything
                sum = __builtin_fmaf(l[e / 4][e % 4], j + e < tile.rank ? (float)x[e] : 0.0f, sum);
        }
        *gptr_w<_Float16>(a.out + row * a.out_row + c) = (_Float16)__builtin_fmaf(sum, tile.scale, (float)*gptr<_Float16>(a.y + row * a.y_row + c));
    }
}

constexpr int kExpandWaves = 4;
constexpr int kLowPad = 8;   // fp16 after each row of low in LDS, against bank conflicts
// Largest ranks of tiles of 16 and of 64 rows, whose low a thread holds in up to 16 and 32
// registers on its way to LDS, beside as many for the parts.  By tiles of 64 and of 16,
// 2048 rows of rank 128 beside 8192 x 8192 take 84.5 and 118 us, of rank 136 by 16 134.
constexpr int kExpandRank16 = 256, kExpandRank64 = 128;

// A wave takes 16 NT columns at a time: NT products whose rows are columns 4 NT q
// + 4 m + i, so that a lane ends up with 4 NT neighbouring columns of one row.
template <int T>
__global__ __launch_bounds__(64 * kExpandWaves, 3) void lora_expand_kernel(LoraArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
    __shared__ float unscale[T];
    constexpr int TT = T / 16, NT = T == 64 ? 2 : 4, COLS = 16 * NT, RANK = T == 64 ? kExpandRank64 : kExpandRank16;
    __shared__ bool lost[T];   // rows for lora_expand_row
    __shared__ __attribute__((aligned(16))) float row_low[kExpandWaves][RANK];
    const int block = blockIdx.x % a.blocks;
    int rows_of_tile;
    const LoraTile tile = lora_tile<T>(a, blockIdx.x / a.blocks, rows_of_tile);
    if (tile.count == 0) return;
    const int t = threadIdx.x, lane = t % 64, wave = t / 64, i16 = lane % 16, q = lane / 16;
    const int n_begin = block * a.columns, n_end = min(a.N, n_begin + a.columns);
    if (tile.adapter < 0) {
        lora_copy(a, tile, rows_of_tile, n_begin, n_end);
        return;
    }
    const int padded = (a.rank + 31) / 32 * 32, pitch = padded + kLowPad;
    uint16_t *hi = lds, *lo = lds + T * pitch;
    // low: a few lanes a row add up its parts, all asked for at once
    constexpr int LANES = 64 * kExpandWaves / T;   // of a row: 16 or 4
    constexpr int MOST = RANK / (4 * LANES);
    const int low_row = t / LANES, first = 4 * (t % LANES);
    const float* from = a.low + (int64_t)__shfl(rows_of_tile, low_row) * a.rank;
    const int64_t part = (int64_t)a.rows * a.rank;
    f4 v[MOST];
#pragma unroll
    for (int m = 0; m < MOST; ++m) {
        const int j = first + 4 * LANES * m;
        v[m] = f4{};
        if (4 * LANES * m >= padded) continue;
        f4 parts[kLoraSplits];
#pragma unroll
        for (int s = 0; s < kLoraSplits; ++s)   // zero behind the adapter's own rank; a.rank is a multiple of 8
            parts[s] = s < a.splits && low_row < tile.count && j < a.rank ? *gptr<f4>(from + s * part + j) : f4{};
#pragma unroll
        for (int s = 0; s < kLoraSplits; ++s) v[m] += parts[s];
    }
    // the wave's first y and B, asked for ahead of their use
    int64_t row[TT];
    bool in[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        in[j] = 16 * j + i16 < tile.count;
        row[j] = __shfl(rows_of_tile, 16 * j + i16);
    }
    const uint16_t* b = a.b + (int64_t)tile.adapter * a.N * a.rank;
    struct Loaded {   // for a step of columns
        h8 y[TT][NT / 2], b[2][NT];
    };
    const auto load_b = [&](Loaded& x, int n0, int k) {   // 64 ranks: whole lines of B where it has as many
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                const int c = n0 + 4 * NT * (i16 / 4) + 4 * m + i16 % 4, j = k + 32 * h + 8 * q;
                x.b[h][m] = c < n_end && j < tile.rank ? *gptr<h8>(b + (int64_t)c * a.rank + j) : h8{};
            }
    };
    const auto load = [&](Loaded& x, int n0) {
        load_b(x, n0, 0);
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int half = 0; half < NT / 2; ++half) {   // N and blocks are multiples of 8
                const int n = n0 + 4 * NT * q + 8 * half;
                x.y[j][half] = in[j] && n < n_end ? *gptr<h8>(a.y + row[j] * a.y_row + n) : h8{};
            }
    };
    Loaded l0, l1;
    load(l0, n_begin + COLS * wave);
    // its largest, and the cut in two: |low| * 2^e below 2^15
    {
        float most = 0.0f;
#pragma unroll
        for (int m = 0; m < MOST; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = __builtin_fabsf(v[m][e]);
                most = x < __builtin_huge_valf() ? __builtin_fmaxf(most, x) : most;
            }
#pragma unroll
        for (int d = 1; d < LANES; d *= 2) most = __builtin_fmaxf(most, __shfl_xor(most, d));
        const int e2 = lora_shift(most);
        bool mine = false;
#pragma unroll
        for (int m = 0; m < MOST; ++m) {
            const int j = first + 4 * LANES * m;
            if (j >= padded) continue;
            h4 h, l;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                _Float16 high, rest;
                lora_cut(v[m][e], e2, high, rest);
                mine = mine || lora_lost(v[m][e], e2);
                h[e] = high;
                l[e] = rest;
            }
            *reinterpret_cast<h4*>(hi + low_row * pitch + j) = h;
            *reinterpret_cast<h4*>(lo + low_row * pitch + j) = l;
        }
        const uint64_t any = __ballot(mine) >> (lane / LANES * LANES) & ((1ull << LANES) - 1);
        if (first == 0) {
            unscale[low_row] = lora_unscale(tile.scale, e2);
            lost[low_row] = any != 0;
        }
    }
    __syncthreads();
    uint64_t lost_rows = __ballot(lane < T && lost[lane % T]);
    float f[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        f[j] = unscale[16 * j + i16];
        in[j] = in[j] && !(lost_rows >> (16 * j + i16) & 1);
    }
    const auto step = [&](Loaded& x, int n0) {
        f4 acc[NT][TT];
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int j = 0; j < TT; ++j) acc[m][j] = f4{};
        for (int k = 0; k < tile.rank; k += 64) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k8 = k + 32 * h + 8 * q;
                if (k + 32 * h >= tile.rank) continue;
                if (k8 + 8 > tile.rank)   // what lies behind the adapter's own rank may be anything
#pragma unroll
                    for (int m = 0; m < NT; ++m)
#pragma unroll
                        for (int e = 0; e < 8; ++e) x.b[h][m][e] = k8 + e < tile.rank ? x.b[h][m][e] : (_Float16)0.0f;
#pragma unroll
                for (int j = 0; j < TT; ++j) {
                    const h8 high = *reinterpret_cast<const h8*>(hi + (16 * j + i16) * pitch + k8);
                    const h8 rest = *reinterpret_cast<const h8*>(lo + (16 * j + i16) * pitch + k8);
#pragma unroll
                    for (int m = 0; m < NT; ++m) {
                        acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x.b[h][m], high, acc[m][j], 0, 0, 0);
                        acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x.b[h][m], rest, acc[m][j], 0, 0, 0);
                    }
                }
            }
            if (k + 64 < tile.rank) load_b(x, n0, k + 64);
        }
        const int n = n0 + 4 * NT * q;
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int half = 0; half < NT / 2; ++half) {
                h8 o;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = (_Float16)__builtin_fmaf(acc[2 * half + e / 4][j][e % 4], f[j], (float)x.y[j][half][e]);
                if (in[j] && n + 8 * half < n_end) *gptr_w<h8>(a.out + row[j] * a.out_row + n + 8 * half) = o;
            }
    };
    // the next step's loads are in flight under this one's products
    constexpr int STEP = COLS * kExpandWaves;
    for (int n0 = n_begin + COLS * wave; n0 < n_end; n0 += 2 * STEP) {
        if (n0 + STEP < n_end) load(l1, n0 + STEP);
        step(l0, n0);
        if (n0 + STEP >= n_end) break;
        if (n0 + 2 * STEP < n_end) load(l0, n0 + 2 * STEP);
        step(l1, n0 + STEP);
    }
    for (; lost_rows; lost_rows &= lost_rows - 1) {   // seldom any
        // (nothing that the loop above would have to keep a register for)
        const int64_t at = a.tile_rows[(int64_t)(blockIdx.x / a.blocks) * T + __builtin_ctzll(lost_rows)];
        const int own = __builtin_amdgcn_readfirstlane(wave), l = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0));
        wave_lds_fence();
        for (int j = l; j < a.rank; j += 64) {
            float x = 0.0f;
            for (int p = 0; p < a.splits; ++p) x += *gptr<float>(a.low + p * part + at * a.rank + j);   // in the order of above
            row_low[own][j] = x;
        }
        wave_lds_fence();
        lora_expand_row(a, tile, at, n_begin + 64 * own + l, n_end, 64 * kExpandWaves, row_low[own]);
    }
}

// All of it for a few rows of small adapters, ranks up to 16: every workgroup takes
// x A^T for itself, K cut over its waves, and a block of columns.  A comes by whole
// lines and is turned into operands in LDS, which a wave has to itself: as operands
// straight from memory, half a line of 16 rows at a time, a CU reads 13 bytes of A a
// clock (K of 8192 12.0 us in a graph, 8.6 so).
constexpr int kAloneWaves = 8, kAloneChunk = 256;   // channels that a wave turns at a time
constexpr int kAlonePitch = kAloneChunk + 8;
constexpr int kAloneColumns = 32 * kAloneWaves;     // of a step

__global__ __launch_bounds__(64 * kAloneWaves) void lora_alone_kernel(LoraArgs a) {
    __shared__ f4 parts[kAloneWaves][64];
    __shared__ __attribute__((aligned(16))) uint16_t turned[kAloneWaves][16 * kAlonePitch];
    const int block = blockIdx.x % a.blocks;
    int rows_of_tile;
    const LoraTile tile = lora_tile_of_few<16>(a, blockIdx.x / a.blocks, rows_of_tile);
    if (tile.count == 0) return;
    const int t = threadIdx.x, lane = t % 64, wave = t / 64, i16 = lane % 16, q = lane / 16;
    const int n_begin = block * a.columns, n_end = min(a.N, n_begin + a.columns);
    if (tile.adapter < 0) {
        lora_copy(a, tile, rows_of_tile, n_begin, n_end);
        return;
    }
    bool in = i16 < tile.count;
    const int64_t row = __shfl(rows_of_tile, i16);
    const uint16_t* b = a.b + (int64_t)tile.adapter * a.N * a.rank;
    struct Loaded {   // for a step of columns, 8 of a row to a lane
        h8 y, b[2];
    };
    const auto load = [&](int n0) {
        Loaded x;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int c = n0 + 8 * (i16 / 4) + 4 * m + i16 % 4, j = 8 * q;
            x.b[m] = c < n_end && j < tile.rank ? *gptr<h8>(b + (int64_t)c * a.rank + j) : h8{};
#pragma unroll
            for (int e = 0; e < 8; ++e) x.b[m][e] = j + e < tile.rank ? x.b[m][e] : (_Float16)0.0f;   // what lies behind may be anything
        }
        const int n = n0 + 8 * q;
        x.y = in && n < n_end ? *gptr<h8>(a.y + row * a.y_row + n) : h8{};
        return x;
    };
    int n0 = n_begin + 32 * wave;
    Loaded next = load(n0);

    const int per = ((a.K + kAloneWaves - 1) / kAloneWaves + 31) / 32 * 32, k_begin = wave * per, k_end = min(a.K, k_begin + per);
    const EXQ_GLOBAL uint16_t *ap = gptr<uint16_t>(a.a + (int64_t)tile.adapter * a.rank * a.K), *xp = gptr<uint16_t>(a.x + row * a.x_row);
    constexpr int STEPS = kAloneChunk / 32;
    struct Chunk {   // two ranks' channels to a load of A, an operand to one of x
        h8 a[8], x[STEPS];
    };
    const auto ask = [&](int k0) {   // K and slices are multiples of 8
        Chunk c;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 2 * i + lane / 32, k = k0 + 8 * (lane % 32);
            c.a[i] = k < k_end && r < tile.rank ? *(const EXQ_GLOBAL h8*)(ap + (int64_t)r * a.K + k) : h8{};
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = k0 + 32 * s + 8 * q;
            c.x[s] = k < k_end && in ? *(const EXQ_GLOBAL h8*)(xp + k) : h8{};
        }
        return c;
    };
    f4 acc{};
    Chunk coming = ask(k_begin);
    for (int k0 = k_begin; k0 < k_end; k0 += kAloneChunk) {
        const Chunk c = coming;
        if (k0 + kAloneChunk < k_end) coming = ask(k0 + kAloneChunk);
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<h8*>(&turned[wave][(2 * i + lane / 32) * kAlonePitch + 8 * (lane % 32)]) = c.a[i];
        wave_lds_fence();
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(*reinterpret_cast<const h8*>(&turned[wave][i16 * kAlonePitch + 32 * s + 8 * q]), c.x[s],
                                                         acc, 0, 0, 0);
        wave_lds_fence();
    }
    parts[wave][lane] = acc;
    __syncthreads();
    // ranks 8 q .. + 7 of row i16, as the second product takes them
    f4 low[2] = {f4{}, f4{}};
    float most = 0.0f;
    if (q < 2) {
#pragma unroll
        for (int w = 0; w < kAloneWaves; ++w)
#pragma unroll
            for (int part = 0; part < 2; ++part) low[part] += parts[w][16 * (2 * q + part) + i16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = __builtin_fabsf(low[e / 4][e % 4]);
            most = x < __builtin_huge_valf() ? __builtin_fmaxf(most, x) : most;
        }
    }
    most = __builtin_fmaxf(most, __shfl_xor(most, 16));
    most = __builtin_fmaxf(most, __shfl_xor(most, 32));
    const int e2 = lora_shift(most);
    h8 high, rest;
    float least = __builtin_huge_valf();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        _Float16 h, l;
        lora_cut(low[e / 4][e % 4], e2, h, l);
        least = __builtin_fminf(least, __builtin_fabsf(low[e / 4][e % 4]));
        high[e] = h;
        rest[e] = l;
    }
    // (the smallest first: zeros aside, which an adapter of fewer ranks has, that is all)
    uint64_t lost_rows = 0;
    if (__ballot(in && 8 * q < tile.rank && __builtin_ldexpf(least, e2) < 0x1p-7f)) {
        bool mine = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) mine = mine || lora_lost(low[e / 4][e % 4], e2);
        lost_rows = __ballot(mine);
        lost_rows = (lost_rows | lost_rows >> 16) & 0xFFFF;
    }
    in = in && !(lost_rows >> i16 & 1);
    const float f = lora_unscale(tile.scale, e2);
    for (; n0 < n_end; n0 += kAloneColumns) {
        const Loaded x = next;
        if (n0 + kAloneColumns < n_end) next = load(n0 + kAloneColumns);
        h8 o;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            f4 sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(x.b[m], high, f4{}, 0, 0, 0);
            sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(x.b[m], rest, sum, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[4 * m + e] = (_Float16)__builtin_fmaf(sum[e], f, (float)x.y[4 * m + e]);
        }
        const int n = n0 + 8 * q;
        if (in && n < n_end) *gptr_w<h8>(a.out + row * a.out_row + n) = o;
    }
    for (; lost_rows; lost_rows &= lost_rows - 1) {   // seldom any
        const int i = __builtin_ctzll(lost_rows);
        float* x = reinterpret_cast<float*>(turned[wave]);
        wave_lds_fence();
        if (q < 2 && i16 == i) {
            *reinterpret_cast<f4*>(x + 8 * q) = low[0];
            *reinterpret_cast<f4*>(x + 8 * q + 4) = low[1];
        }
        wave_lds_fence();
        lora_expand_row(a, tile, __builtin_amdgcn_readlane(rows_of_tile, i), n_begin + t, n_end, 64 * kAloneWaves, x);
    }
}

}  // namespace exq

// =================================================================== host

using namespace exq;

namespace {

// Shape of a call.
struct LoraPlan {
    LoraGroup group;
    bool alone;   // in one launch
    int tile_rows, tiles, splits, slice, rank_tiles;
    size_t rows_at, place_at, low_at, bytes;   // of the workspace
};

exq_status plan_lora(const exq_adapters* h, int rows, LoraPlan* p) {
    if (!h) return fail(EXQ_ERR_INVALID_ARG, "adapters is NULL");
    if (rows < 0) return fail(EXQ_ERR_INVALID_ARG, "rows=%d", rows);
    *p = LoraPlan{};
    if (rows == 0) return EXQ_OK;
    p->tile_rows = rows >= 512 && h->rank <= kExpandRank64 ? 64 : 16;
    p->group = rows <= kLoraFew ? kByWave
               : rows <= kLoraSome && h->count + 2 <= 64 * shrink_waves(p->tile_rows) ? kByWorkgroup : kByLaunch;
    p->tiles = (int)std::min<int64_t>(rows, (int64_t)rows / p->tile_rows + h->count + 2);
    p->rank_tiles = h->rank <= 16 ? 1 : h->rank <= 32 || p->group == kByWave ? 2 : 4;
    // Two launches and one, in a graph (us): K and N of 1024 and 4096 7.9, 5.2; 4096 8.2, 6.5, 8 rows 9.1, 7.4; 8192
    // 8.4, 8.6, 4 rows 8.9, 9.7.  A call costs the host 8 and 4.4 us.
    p->alone = h->rank <= 16 && (rows <= 2 ? h->K <= 8192 : rows <= 16 && h->K <= 4096);
    if (p->alone) return EXQ_OK;
    // a wave's channels are all in flight at once, or there are four waves a SIMD
    // already: workgroups that wait for a place would double the time (2048 rows of
    // 8192 in 4 parts, 280 workgroups, 21 us, in 3 parts 18.5)
    const int rank_blocks = (h->rank + 16 * p->rank_tiles - 1) / (16 * p->rank_tiles);
    const int W = shrink_waves(p->tile_rows), TT = shrink_rows(p->tile_rows);
    const int channels = 32 * W * (p->rank_tiles == 4 && TT == 2 ? kShrinkSteps<2, 4> : kShrinkSteps<1, 1>);
    const int most = std::min(kLoraSplits, (h->K + channels - 1) / channels);
    const int64_t part_tiles = ((int64_t)rows + 16 * TT - 1) / (16 * TT) + (TT > 1 ? std::min(h->count, rows / 64) : 0);   // half of them filled
    p->splits = (int)std::max<int64_t>(1, std::min<int64_t>(most, 4096 / W / (part_tiles * rank_blocks)));
    const int unit = 32 * W;
    p->slice = ((h->K + p->splits - 1) / p->splits + unit - 1) / unit * unit;
    p->splits = (h->K + p->slice - 1) / p->slice;
    p->rows_at = sizeof(LoraTile) * (size_t)p->tiles;
    p->place_at = p->rows_at + 4 * (size_t)p->tiles * p->tile_rows;
    p->low_at = (p->place_at + (rows > kLoraGroupThreads * kLoraGroupEach ? 4 * (size_t)rows : 0) + 15) / 16 * 16;
    p->bytes = p->low_at + 4 * (size_t)p->splits * rows * h->rank;
    return EXQ_OK;
}

template <LoraGroup GROUP, int T> exq_status launch_lora(const LoraArgs& a, const LoraPlan& p, hipStream_t s) {
    exq_status st;
    if (GROUP == kByLaunch) {
        hipLaunchKernelGGL(lora_group_kernel, dim3(1), dim3(kLoraGroupThreads), 0, s, a, T, p.tiles);
        if ((st = launched("adapters group launch")) != EXQ_OK) return st;
    }
    const int ranks = 16 * p.rank_tiles;
    const dim3 grid((unsigned)(p.tiles * (T / 16 / shrink_rows(T)) * p.splits), (unsigned)((a.rank + ranks - 1) / ranks));
    const dim3 block(64 * shrink_waves(T));
    if (p.rank_tiles == 1) hipLaunchKernelGGL((lora_shrink_kernel<GROUP, T, 1>), grid, block, 0, s, a);
    else if (GROUP == kByWave || p.rank_tiles == 2) hipLaunchKernelGGL((lora_shrink_kernel<GROUP, T, 2>), grid, block, 0, s, a);
    else if constexpr (GROUP != kByWave) hipLaunchKernelGGL((lora_shrink_kernel<GROUP, T, 4>), grid, block, 0, s, a);
    if ((st = launched("adapters shrink launch")) != EXQ_OK) return st;
    const int pitch = (a.rank + 31) / 32 * 32 + kLowPad;
    hipLaunchKernelGGL((lora_expand_kernel<T>), dim3((unsigned)(p.tiles * a.blocks)), dim3(64 * kExpandWaves), 2u * 2u * T * pitch, s, a);
    return launched("adapters expand launch");
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
    if (p.bytes && (!workspace || !aligned(workspace, 16) || workspace_bytes < p.bytes))
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
    a.tiles = reinterpret_cast<LoraTile*>(ws);
    a.tile_rows = reinterpret_cast<int32_t*>(ws + p.rows_at);
    a.place = reinterpret_cast<int32_t*>(ws + p.place_at);
    a.low = reinterpret_cast<float*>(ws + p.low_at);
    a.splits = p.splits;
    a.slice = p.slice;
    a.in_place = in_place;
    if (p.alone) {
        const int steps = (h->N + kAloneColumns - 1) / kAloneColumns;
        a.columns = kAloneColumns * std::max(1, (int)((int64_t)steps * std::min(p.tiles, h->count + 1) / 256));
        a.blocks = (h->N + a.columns - 1) / a.columns;
        const hipStream_t s = static_cast<hipStream_t>(stream);
        const dim3 grid((unsigned)(p.tiles * a.blocks)), block(64 * kAloneWaves);
        hipLaunchKernelGGL(lora_alone_kernel, grid, block, 0, s, a);
        return launched("adapters launch");
    }
    // blocks that make at most about 750 workgroups, which run side by side
    const int unit = 16 * (p.tile_rows == 64 ? 2 : 4) * kExpandWaves, units = (h->N + unit - 1) / unit;
    const int busy = p.group == kByWave ? std::min(rows, h->count + 1) : std::min(p.tiles, rows / p.tile_rows + 1);
    a.columns = unit * (int)std::min<int64_t>(units, ((int64_t)units * busy + 749) / 750);
    a.blocks = (h->N + a.columns - 1) / a.columns;
    if ((int64_t)p.tiles * std::max(a.blocks, p.splits * (p.tile_rows / 16)) > kMaxLaunchThreads / 512)
        return fail(EXQ_ERR_UNSUPPORTED, "%d rows in one call", rows);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (p.group == kByWave) return launch_lora<kByWave, 16>(a, p, s);
    if (p.group == kByWorkgroup) return p.tile_rows == 64 ? launch_lora<kByWorkgroup, 64>(a, p, s) : launch_lora<kByWorkgroup, 16>(a, p, s);
    return p.tile_rows == 64 ? launch_lora<kByLaunch, 64>(a, p, s) : launch_lora<kByLaunch, 16>(a, p, s);
}

}  // extern "C"
