// Paged key-value cache of libexq for gfx950: quantized append, read-back, and
// attention of one new token over it.  include/exq.h documents the layout;
// every kernel here reads or writes it directly.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "exq_device_common.h"
#include "exq_internal.h"

// Geometry of a cache and its borrowed pages (the exq_cache_t handle).
struct exq_cache {
    uint8_t* pages;
    int64_t n_pages;
    int page_size, kv_heads, head_dim, k_bits, v_bits;
    size_t page_bytes;
};

namespace exq {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int kCacheTile = 16;    // tokens per tile
constexpr int kCacheGroup = 32;   // channels per scale
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Bytes of one part (codes, then scales) of a tile, and the byte in the code
// part of lane l's b-byte unit of group g (see the layout in include/exq.h).
template <int D, int B> struct CachePart {
    static constexpr int G = D / kCacheGroup;
    static constexpr int GPC = 16 / B;                            // groups per full chunk
    static constexpr int CHUNKS = (G + GPC - 1) / GPC;
    static constexpr int CODES = kCacheTile * D * B / 8;
    static constexpr int SCALES = B < 16 ? kCacheTile * G * 2 : 0;
    static constexpr int BYTES = CODES + SCALES;
    __device__ static constexpr int chunk_groups(int j) { return G - j * GPC < GPC ? G - j * GPC : GPC; }
    __device__ static int unit(int lane, int g) {
        const int j = g / GPC;
        return 1024 * j + lane * (chunk_groups(j) * B) + (g - j * GPC) * B;
    }
};

// Bytes of one token of one head.
constexpr int row_bytes(int head_dim, int k_bits, int v_bits) {
    const int scales = 2 * (head_dim / kCacheGroup);
    return head_dim * k_bits / 8 + head_dim * v_bits / 8 + (k_bits < 16 ? scales : 0) + (v_bits < 16 ? scales : 0);
}

// What the kernels know about a cache.
struct CacheDev {
    uint8_t* pages;
    int64_t page_bytes;
    uint32_t n_pages, page_size, kv_heads;
    uint32_t tiles;   // per page and head
};

struct TableDev {
    const int32_t* pages;
    int64_t stride;
    uint32_t rows, width;
};

// The fp16 values of a lane's eight elements of a group: x_hat = (c - z) * s,
// the difference exact in fp16, the product rounded once.  W: the unit's
// B / 4 dwords; s0, s1: the scales of halves 0 and 1 of a pair (keys: the
// token's, twice; values: tokens 0, 1, and s2, s3 for tokens 2, 3).
__device__ __forceinline__ uint32_t scaled(uint32_t biased, uint32_t zero, uint32_t s) {
    const h2 v = (as_h2(biased) - as_h2(zero)) * as_h2(s);
    return __builtin_bit_cast(uint32_t, v);
}

// 0x6400 is fp16 1024, whose last bit is worth 1: an integer code below 1024
// OR-ed into it gives 1024 + c.
template <int B> constexpr uint32_t kBiasedZero = B == 4 ? 0x64086408u : 0x64806480u;   // 1024 + 2^(B-1)

__device__ __forceinline__ uint32_t nibbles(uint32_t w) { return (w & 0x000F000Fu) | 0x64006400u; }

// Constants of the 4-bit decoding in registers.  The compiler is not shown
// their values: it would rather write a mask and the 0x6400 as literals of two
// instructions than as registers of one v_and_or_b32.
struct Nibbles {
    uint32_t even, odd, one_even, one_odd;
    __device__ __forceinline__ void init() {
        even = 0x000F000Fu;
        odd = 0x00F000F0u;
        one_even = 0x64006400u;   // fp16 1024, whose bit 0 is worth 1
        one_odd = 0x54005400u;    // fp16 64, whose bit 4 is worth 1
        asm volatile("" : "+v"(even), "+v"(odd), "+s"(one_even), "+s"(one_odd));
    }
    // The pair of codes at bits 4 e and 4 e + 16 of w, less 8, exactly; one
    // shift by 8 serves e = 2 and 3.
    template <int E> __device__ __forceinline__ h2 pair(uint32_t w) const {
        const uint32_t x = E >= 2 ? w >> 8 : w;
        if constexpr (E % 2 == 0) return as_h2((x & even) | one_even) - h2{1032, 1032};
        else return as_h2((x & odd) | one_odd) - h2{72, 72};
    }
};

// ------------------------------------------------------------------ append

// Where row r goes: its tile's first byte (of head 0) and token in the tile.
// at < 0: nowhere (-1 padding, -2 outside the table or the cache).
struct RowPlace {
    int64_t at;
    int token;
};

// Row r's place (r < 0: none); ahead(): loads to ask for once the page's is.
template <class F>
__device__ __forceinline__ RowPlace row_place(const CacheDev& c, const TableDev& t, const int32_t* seqs,
                                              const int32_t* positions, int r, int tile_bytes, F&& ahead) {
    const int32_t s = r >= 0 ? gptr<int32_t>(seqs)[r] : -1, p = r >= 0 ? gptr<int32_t>(positions)[r] : 0;
    const uint32_t pi = (uint32_t)p / c.page_size, in = (uint32_t)p % c.page_size;
    const bool inside = s >= 0 && (uint32_t)s < t.rows && p >= 0 && pi < t.width;
    const uint32_t page = inside ? (uint32_t)gptr<int32_t>(t.pages)[(int64_t)s * t.stride + pi] : 0u;
    ahead();
    if (s < 0) return {-1, 0};
    if (!inside || page >= c.n_pages) return {-2, 0};
    return {(int64_t)page * c.page_bytes + (int64_t)(in / kCacheTile) * tile_bytes, (int)(in % kCacheTile)};
}

// Append and read run one wave for 16 rows of one head: lane 16 q + t holds
// channels 32 g + 8 q + (0..7) of every group g of row t, which is the keys'
// own unit in the cache, so a lane moves its keys to or from wherever its row
// lies, and 16 rows that fill a tile move as one contiguous run.  Values are
// laid out by channel and have to change lanes: through LDS where the 16 rows
// are a tile, by bytes where they are not.  Blocks of rows start where the
// first row's tile starts, so that one sequence's rows (a prompt) make tiles
// wherever the prompt starts.  A second sequence's rows make tiles only if they
// happen to be in step with them: 8 prompts of 1001 tokens and 8 heads in one call
// at 4 bits are appended in 16.3 us and read in 22, one of 8008 in 12 and 9 (in 16
// bits 22.6 and 24, 10.6 and 12).
constexpr int kRowsThreads = 256;

// Orders a wave's own LDS writes before its reads, and its reads before its
// next writes.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The rows of a lane and where they lie.
struct RowsBlock {
    int row, head;     // row < 0: none
    RowPlace place;
    bool tile;         // the wave's 16 rows are the 16 tokens of one tile, in order
};

// ahead(b): loads that do not wait for the rows' places.
template <class F>
__device__ __forceinline__ RowsBlock rows_block(const CacheDev& c, const TableDev& t, const int32_t* seqs,
                                                const int32_t* positions, int rows, int tile_bytes, F&& ahead) {
    RowsBlock b;
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t i = (int64_t)blockIdx.x * (kRowsThreads / 64) + wave;
    b.head = (int)(i % c.kv_heads);
    const int64_t r = i / c.kv_heads * kCacheTile - (gptr<int32_t>(positions)[0] & (kCacheTile - 1)) + (lane & 15);
    b.row = r >= 0 && r < rows ? (int)r : -1;
    b.place = row_place(c, t, seqs, positions, b.row, tile_bytes, [&] { ahead(b); });
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b.place.at);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)b.place.at >> 32));
    const bool same = b.place.at >= 0 && b.place.token == (lane & 15) && (uint64_t)b.place.at == (((uint64_t)hi << 32) | lo);
    b.tile = __builtin_amdgcn_ballot_w64(same) == ~0ull;
    return b;
}

// max|x| of each group over the lane's 8 channels, then over the 4 lanes of
// its row, as fp16 bits: ordered like integers, infinities and NaN on top.
// Two groups to a dword.
template <int G>
__device__ __forceinline__ void group_max(const u4v (&x)[G], uint32_t (&m)[(G + 1) / 2]) {
    typedef uint16_t us2 __attribute__((ext_vector_type(2)));
    auto top = [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b)));
    };
    uint32_t h[G + 1];
    h[G] = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint32_t a = x[g][0] & 0x7FFF7FFFu, b = x[g][1] & 0x7FFF7FFFu, c = x[g][2] & 0x7FFF7FFFu, d = x[g][3] & 0x7FFF7FFFu;
        h[g] = top(top(a, b), top(c, d));
    }
#pragma unroll
    for (int i = 0; i < (G + 1) / 2; ++i) {
        // low halves of both groups against their high halves
        const uint32_t a = h[2 * i], b = h[2 * i + 1];
        uint32_t v = top((a & 0xFFFFu) | (b << 16), (a >> 16) | (b & 0xFFFF0000u));
        v = top(v, (uint32_t)__shfl_xor((int)v, 16));
        v = top(v, (uint32_t)__shfl_xor((int)v, 32));
        m[i] = v;
    }
}

// A group's scale from its max|x|: fp16 bits.  The quotient by 7 or 127, one
// Newton step on m * (1 / top): no quotient of an 11-bit number by these lies
// within 2^-46 of a tie of fp32, so it is the correctly rounded one.  At most
// the largest scale whose largest code's value, top * s, is finite in fp16
// (the next ones give 65520 and 65532, which round to infinity).
template <int B> __device__ __forceinline__ uint32_t scale_bits(uint32_t max_bits) {
    constexpr float top = (float)((1 << (B - 1)) - 1), inv = 1.0f / top, most = B == 4 ? 9352.0f : 515.5f;
    const float m = (float)__builtin_bit_cast(_Float16, (uint16_t)max_bits);
    const float q0 = m * inv, q = __builtin_fmaf(__builtin_fmaf(-q0, top, m), inv, q0);
    return max_bits >= 0x7C00u ? 0x7E00u : (uint32_t)f32_to_f16_bits(__builtin_fminf(q, most));
}

// Codes of eight values at scale s.  The quotient x / s: one Newton step on
// x * (1 / s) leaves it within 2^-44 of itself before its rounding to fp32, so
// a quotient that lies on a tie (k + 1/2, which fp32 holds) comes out exact,
// and any other lies at least 2^-12 from a tie (s has 11 bits).  Adding 1.5 *
// 2^23 + z rounds it to the nearest integer, ties to even, and leaves the code
// in the sum's low bits.
template <int B> __device__ __forceinline__ void codes_of(const u4v& x, uint32_t s_bits, uint32_t (&c)[8]) {
    constexpr float top = (float)((1 << (B - 1)) - 1), magic = 12582912.0f + (float)(1 << (B - 1));
    const float s = (float)__builtin_bit_cast(_Float16, (uint16_t)s_bits);
    // zero scale: every quotient 0; NaN scale: codes that say nothing
    const float inv = s > 0.0f ? __builtin_amdgcn_rcpf(s) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t w = x[e / 2];
        const float f = (float)as_h2(w)[e % 2];
        const float q0 = f * inv, q = __builtin_fmaf(__builtin_fmaf(-q0, s, f), inv, q0);
        c[e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(q, -top, top) + magic) & ((1u << B) - 1u);
    }
}

// Four nibbles of the low half of x, one to a byte.
__device__ __forceinline__ uint32_t spread(uint32_t x) {
    uint32_t t = x & 0xFFFFu;
    t = (t | (t << 8)) & 0x00FF00FFu;
    return (t | (t << 4)) & 0x0F0F0F0Fu;
}

// Bound by the bytes of k and v in and of the codes out: 16384 rows of 8 heads
// of 128 at 4 bits (67 MB in, 19 out) 20-25 us, 3.4-4.3 TB/s of a copy's 4.8.
template <int D, int KB, int VB>
__global__ __launch_bounds__(kRowsThreads) void append_kernel(CacheDev c, TableDev t, const uint16_t* __restrict__ k,
                                                              int64_t k_row, int64_t k_head,
                                                              const uint16_t* __restrict__ v, int64_t v_row,
                                                              int64_t v_head, int rows,
                                                              const int32_t* __restrict__ seqs,
                                                              const int32_t* __restrict__ positions) {
    using PK = CachePart<D, KB>;
    using PV = CachePart<D, VB>;
    constexpr int G = D / kCacheGroup, TILE = PK::BYTES + PV::BYTES;
    __shared__ __attribute__((aligned(16))) uint8_t turned[kRowsThreads / 64][PV::CODES];
    const int lane = (int)threadIdx.x & 63, q = lane >> 4;
    u4v kx[G], vx[G];
    const RowsBlock b = rows_block(c, t, seqs, positions, rows, TILE, [&](const RowsBlock& b) {
        const int64_t r = b.row >= 0 ? b.row : 0;
        const uint16_t *ks = k + r * k_row + b.head * k_head + 8 * q, *vs = v + r * v_row + b.head * v_head + 8 * q;
#pragma unroll
        for (int g = 0; g < G; ++g) kx[g] = *gptr<u4v>(ks + g * kCacheGroup);
#pragma unroll
        for (int g = 0; g < G; ++g) vx[g] = *gptr<u4v>(vs + g * kCacheGroup);
    });
    if (__builtin_amdgcn_ballot_w64(b.place.at >= 0) == 0) return;
    uint8_t* buf = turned[threadIdx.x >> 6];
    uint8_t* tile = c.pages + (b.place.at >= 0 ? b.place.at : 0) + (int64_t)b.head * c.tiles * TILE;
    const bool live = b.place.at >= 0;
    const int tok = b.place.token;

    // keys
    if constexpr (KB == 16) {
        if (live) {
#pragma unroll
            for (int g = 0; g < G; ++g) *gptr_w<u4v>(tile + PK::unit(16 * q + tok, g)) = kx[g];
        }
    } else {
        uint32_t m[(G + 1) / 2], w[G * KB / 4], s[G];
        group_max<G>(kx, m);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            s[g] = scale_bits<KB>((m[g / 2] >> (16 * (g % 2))) & 0xFFFFu);
            uint32_t code[8];
            codes_of<KB>(kx[g], s[g], code);
            if constexpr (KB == 4) {
                uint32_t x = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) x |= code[e] << (4 * (e / 2) + 16 * (e % 2));
                w[g] = x;
            } else {
                w[2 * g] = code[0] | (code[1] << 8) | (code[2] << 16) | (code[3] << 24);
                w[2 * g + 1] = code[4] | (code[5] << 8) | (code[6] << 16) | (code[7] << 24);
            }
        }
        if (live) {
            static_for<0, PK::CHUNKS>([&](auto jc) {
                constexpr int j = jc, n = (G - j * PK::GPC < PK::GPC ? G - j * PK::GPC : PK::GPC) * KB / 4;
                uint8_t* dst = tile + 1024 * j + (16 * q + tok) * (4 * n);
                if constexpr (n == 4) *gptr_w<u4v>(dst) = u4v{w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]};
                else {
#pragma unroll
                    for (int i = 0; i < n; ++i) gptr_w<uint32_t>(dst)[i] = w[4 * j + i];
                }
            });
            if (q == 0) {
#pragma unroll
                for (int g = 0; g < G; ++g) gptr_w<uint16_t>(tile + PK::CODES + 2 * tok * G)[g] = (uint16_t)s[g];
            }
        }
    }

    // values: the bytes (16 bits: halves) of the lane's channels, two (four)
    // dwords a group
    uint8_t* part = tile + PK::BYTES;
    const int t4 = tok % 4, half = q / 2;
    constexpr int WORDS = VB == 16 ? 4 : 2;
    uint32_t w[G][WORDS];
    if constexpr (VB == 16) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[g][i] = vx[g][i];
    } else {
        uint32_t m[(G + 1) / 2], s[G];
        group_max<G>(vx, m);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            s[g] = scale_bits<VB>((m[g / 2] >> (16 * (g % 2))) & 0xFFFFu);
            uint32_t c8[8];
            codes_of<VB>(vx[g], s[g], c8);
            if constexpr (VB == 4) {
                // channels c and c + 16 share a byte: lanes q = 2, 3 hand theirs to q = 0, 1
                uint32_t x = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) x |= c8[e] << (4 * e);
                const uint32_t y = (uint32_t)__shfl_xor((int)x, 32);
                w[g][0] = spread(x) | (spread(y) << 4);
                w[g][1] = spread(x >> 16) | (spread(y >> 16) << 4);
            } else {
                w[g][0] = c8[0] | (c8[1] << 8) | (c8[2] << 16) | (c8[3] << 24);
                w[g][1] = c8[4] | (c8[5] << 8) | (c8[6] << 16) | (c8[7] << 24);
            }
        }
        // (a row's four lanes hold the same scales: lane q = 0 stores them)
        if (live && q == 0) {
#pragma unroll
            for (int g = 0; g < G; ++g)
                gptr_w<uint16_t>(part + PV::CODES + 8 * G * (tok / 4) + 2 * t4)[4 * g] = (uint16_t)s[g];
        }
    }
    // Element e of group g goes to the unit of lane 16 (tok / 4) + 8 (q % 2) + e.
    const int unit_lane = 16 * (tok / 4) + 8 * (q % 2);
    const int inner = VB == 4 ? 2 * (t4 % 2) + t4 / 2 : VB == 8 ? 4 * half + t4 : 8 * half + 2 * t4;
    auto scatter = [&](auto put) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = PV::unit(unit_lane, g) + e * (PV::chunk_groups(g / PV::GPC) * VB) + inner;
                put(at, VB == 16 ? w[g][e / 2] >> (16 * (e % 2)) : w[g][e / 4] >> (8 * (e % 4)));
            }
    };
    const bool mine = live && (VB != 4 || half == 0);
    if (b.tile) {
        if (mine) {
            scatter([&](int at, uint32_t x) {
                if constexpr (VB == 16) *reinterpret_cast<uint16_t*>(buf + at) = (uint16_t)x;
                else buf[at] = (uint8_t)x;
            });
        }
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < (PV::CODES + 1023) / 1024; ++i) {
            const int at = 1024 * i + 16 * lane;
            if (PV::CODES % 1024 == 0 || at < PV::CODES) *gptr_w<u4v>(part + at) = *reinterpret_cast<const u4v*>(buf + at);
        }
    } else if (mine) {
        scatter([&](int at, uint32_t x) {
            if constexpr (VB == 16) *gptr_w<uint16_t>(part + at) = (uint16_t)x;
            else *gptr_w<uint8_t>(part + at) = (uint8_t)x;
        });
    }
}

// -------------------------------------------------------------------- read

// Bound by the fp16 rows out: 32768 rows of 8 heads of 128 at 4 bits (38 MB in,
// 134 out) 31-36 us, 4.8-5.6 TB/s of a copy's 4.8.
template <int D, int KB, int VB>
__global__ __launch_bounds__(kRowsThreads) void cache_read_kernel(CacheDev c, TableDev t, uint16_t* __restrict__ k,
                                                                  int64_t k_row, int64_t k_head,
                                                                  uint16_t* __restrict__ v, int64_t v_row,
                                                                  int64_t v_head, int rows,
                                                                  const int32_t* __restrict__ seqs,
                                                                  const int32_t* __restrict__ positions) {
    using PK = CachePart<D, KB>;
    using PV = CachePart<D, VB>;
    constexpr int G = D / kCacheGroup, TILE = PK::BYTES + PV::BYTES, PITCH = D + 8;
    __shared__ __attribute__((aligned(16))) uint16_t turned[kRowsThreads / 64][kCacheTile][PITCH];
    const RowsBlock b = rows_block(c, t, seqs, positions, rows, TILE, [](const RowsBlock&) {});
    if (__builtin_amdgcn_ballot_w64(b.place.at != -1) == 0) return;
    const int lane = (int)threadIdx.x & 63, q = lane >> 4;
    const bool live = b.place.at >= 0, written = b.place.at != -1;
    const int tok = live ? b.place.token : 0;
    const uint8_t* tile = c.pages + (live ? b.place.at : 0) + (int64_t)b.head * c.tiles * TILE;   // rows outside read tile 0
    const uint8_t* part = tile + PK::BYTES;
    uint16_t (&buf)[kCacheTile][PITCH] = turned[threadIdx.x >> 6];
    const u4v nan = {0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u};

    // what there is to load, all at once
    uint32_t kw[G * KB / 4], ksc[(G + 1) / 2], vw[G * VB / 4], vsc[2 * G];
    auto load_unit_words = [&](auto bits, uint32_t* w, const uint8_t* src, int unit_lane) {
        constexpr int B = bits;
        using P = CachePart<D, B>;
        static_for<0, P::CHUNKS>([&](auto jc) {
            constexpr int j = jc, n = (G - j * P::GPC < P::GPC ? G - j * P::GPC : P::GPC) * B / 4;
            const uint8_t* at = src + 1024 * j + unit_lane * (4 * n);
            if constexpr (n == 4) {
                const u4v x = *gptr<u4v>(at);
                w[4 * j] = x[0]; w[4 * j + 1] = x[1]; w[4 * j + 2] = x[2]; w[4 * j + 3] = x[3];
            } else {
#pragma unroll
                for (int i = 0; i < n; ++i) w[4 * j + i] = gptr<uint32_t>(at)[i];
            }
        });
    };
    load_unit_words(IC<KB>{}, kw, tile, 16 * q + tok);
    if constexpr (KB < 16) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const uint32_t s = gptr<uint16_t>(tile + PK::CODES + 2 * tok * G)[g];
            ksc[g / 2] = g % 2 ? ksc[g / 2] | (s << 16) : s;
        }
    }
    if (b.tile) {
        load_unit_words(IC<VB>{}, vw, part, lane);
        if constexpr (VB < 16) {
#pragma unroll
            for (int i = 0; i < 2 * G; ++i) vsc[i] = gptr<uint32_t>(part + PV::CODES + 8 * G * q)[i];
        }
    }

    // keys: the lane's own channels
    uint16_t *kd = k + (int64_t)(written ? b.row : 0) * k_row + b.head * k_head + 8 * q;
    uint16_t *vd = v + (int64_t)(written ? b.row : 0) * v_row + b.head * v_head + 8 * q;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        u4v o;
        if constexpr (KB == 16) {
            o = u4v{kw[4 * g], kw[4 * g + 1], kw[4 * g + 2], kw[4 * g + 3]};
        } else {
            const uint32_t s = ((ksc[g / 2] >> (16 * (g % 2))) & 0xFFFFu) * 0x10001u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (KB == 4) {
                    o[e] = scaled(nibbles(kw[g] >> (4 * e)), kBiasedZero<4>, s);
                } else {
                    const uint32_t w = kw[2 * g + e / 2] >> (16 * (e % 2));
                    o[e] = scaled((w & 0xFFu) | ((w & 0xFF00u) << 8) | 0x64006400u, kBiasedZero<8>, s);
                }
            }
        }
        if (b.tile) *reinterpret_cast<u4v*>(&buf[lane & 15][kCacheGroup * g + 8 * q]) = o;
        else if (written) *gptr_w<u4v>(kd + g * kCacheGroup) = live ? o : nan;
    }

    // A tile's rows leave as whole rows, one after the other: written from the
    // lanes that hold them, in runs of 64 bytes, 32768 rows at 4 bits took 45 us
    // and now take 37.
    auto store_tile = [&](uint16_t* dst, int64_t row_stride, int64_t head_stride) {
        wave_lds_fence();
        uint16_t* first = dst + (int64_t)(b.row - (lane & 15)) * row_stride + b.head * head_stride;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int at = 64 * i + lane, r = at / (D / 8), d = at % (D / 8) * 8;
            *gptr_w<u4v>(first + r * row_stride + d) = *reinterpret_cast<const u4v*>(&buf[r][d]);
        }
        wave_lds_fence();
    };

    // values
    if (b.tile) {
        store_tile(k, k_row, k_head);
        // the lane's four tokens of channels 32 g + col and 32 g + 16 + col, turned in the wave's own LDS
        const int col = lane & 15;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t x[2];   // tokens 4 q, 4 q + 1 and 4 q + 2, 4 q + 3
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if constexpr (VB == 16) {
                        x[i] = vw[4 * g + 2 * h + i];
                    } else if constexpr (VB == 4) {
                        x[i] = scaled(nibbles(vw[g] >> (4 * h + 8 * i)), kBiasedZero<4>, vsc[2 * g + i]);
                    } else {
                        const uint32_t w = vw[2 * g + h] >> (16 * i);
                        x[i] = scaled((w & 0xFFu) | ((w & 0xFF00u) << 8) | 0x64006400u, kBiasedZero<8>, vsc[2 * g + i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    buf[4 * q + i][kCacheGroup * g + 16 * h + col] = (uint16_t)(i % 2 ? x[i / 2] >> 16 : x[i / 2]);
            }
        store_tile(v, v_row, v_head);
    } else if (written) {
        const int t4 = tok % 4, col0 = 8 * (q % 2), half = q / 2;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint32_t s = 0;
            if constexpr (VB < 16)
                s = (uint32_t)*gptr<uint16_t>(part + PV::CODES + 8 * G * (tok / 4) + 8 * g + 2 * t4) * 0x10001u;
            u4v o;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t x[2];
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const uint8_t* u = part + PV::unit(16 * (tok / 4) + col0 + 2 * e + f, g);
                    if constexpr (VB == 16) x[f] = gptr<uint16_t>(u)[4 * half + t4];
                    else if constexpr (VB == 8) x[f] = gptr<uint8_t>(u)[4 * half + t4];
                    else x[f] = ((uint32_t)gptr<uint8_t>(u)[2 * (t4 % 2) + t4 / 2] >> (4 * half)) & 15u;
                }
                const uint32_t w = x[0] | (x[1] << 16);
                if constexpr (VB == 16) o[e] = w;
                else o[e] = scaled(w | 0x64006400u, kBiasedZero<VB>, s);
            }
            *gptr_w<u4v>(vd + g * kCacheGroup) = live ? o : nan;
        }
    }
}

// ------------------------------------------------------------------ attend

constexpr int kCusLog2 = 8, kCus = 1 << kCusLog2;
// Calls of more segments or rows are not split.  Equal rows load the card
// evenly as they are (300 rows of 500 tokens and 8 heads at 4 bits 42 us), but
// a long one among them runs alone in a workgroup a head: with one of 131072
// tokens the 300 rows take 1106 us, where 255 with the same one, split, take
// 70; 128 rows of 32 heads with one of 32768 take 294.
constexpr int kAttendMaxSegments = 2048;
constexpr int kAttendMaxRows = 256;
// Parts of a segment: 8 segments have one for each CU.  Fewer leave CUs idle:
// 131072 tokens at 4 bits take 34 us with 8 key-value heads, and 32, 30 and 28
// with 4, 2 and 1.
constexpr int kAttendMaxParts = 32;
constexpr int kAttendMaxWgs = kAttendMaxSegments + 2 * kCus;   // of a launch that splits
constexpr int kJoinBatch = 16;             // parts whose loads a thread has in flight at once

// Waves per SIMD a geometry's kernel is compiled for: as many as its raw data,
// query and sums leave registers for.
constexpr int attend_waves_per_simd(int D, int KB, int VB) {
    return D <= 96 ? 4 : D == 128 ? (KB + VB <= 8 ? 4 : 3) : KB + VB <= 16 ? 2 : 1;
}

// Geometries that have a kernel of 8 waves a workgroup beside the one of 4.
constexpr bool attend_light(int D, int KB, int VB) { return row_bytes(D, KB, VB) <= 208; }

// Geometries of 4 bits for which four workgroups a CU may pay, and fit.
constexpr bool attend_full(int D, int KB, int VB) { return D % 64 == 0 && KB + VB == 8 && attend_waves_per_simd(D, KB, VB) == 4; }

// The workspace starts with the arrival counters of segments (at their first
// workgroup's number), zero between launches.
constexpr size_t kCounterBytes = EXQ_ATTEND_COUNTER_BYTES;
static_assert(kCounterBytes >= kAttendMaxWgs * sizeof(uint32_t), "a counter for every workgroup");

// Division of a 32-bit number by d with one product: m = floor(2^32 / d) + 1
// gives a quotient that is at most one too high (m = 0 stands for d = 1).
struct Divisor {
    uint32_t d, m;
    __host__ static Divisor of(uint32_t d) { return {d, d == 1 ? 0u : (uint32_t)((1ull << 32) / d + 1)}; }
    __device__ __forceinline__ uint32_t divide(uint32_t n) const {
        const uint32_t q = m ? __umulhi(n, m) : n;
        return q * d > n ? q - 1 : q;
    }
};

// Longest row: tokens are counted in 32 bits, up to a few units past the end.
constexpr int kMaxLength = 0x7FFF0000;

struct AttendArgs {
    CacheDev c;
    TableDev t;
    const uint16_t* q;
    int64_t q_row, q_head;
    uint16_t* out;
    int64_t out_row, out_head;
    float* lse;                // may be null
    const int32_t* lengths;
    float* ws;
    float scale;               // scale * log2(e)
    int window;
    int most;                  // longest row: what the table holds, kMaxLength at most
    int rows, q_heads, group;  // group: query heads per key-value head
    Divisor head_tiles;        // kv_heads * ceil(group / 16): segments of a row
    Divisor group_tiles;       // ceil(group / 16)
    Divisor page_tiles;        // tiles of a page and head
    int whole_units;           // rows of at most this many units are not split
    int target;                // log2 of the workgroups to split for; 0: a workgroup for each segment
    int other;                 // log2 of another number of workgroups, for lengths that come out at no more; 0: none
    int other_size;            // if chunks would have at least so many units then,
    float other_rows;          // and the rows together are as long as so many of the longest
    int slack;                 // twelfths by which chunks may be longer for it
};

// Tokens [lo, hi) that a row of length n attends to, and its number of units
// of `unit` tokens from the one that holds lo.  Rows left alone have no unit;
// empty rows and rows to be filled with NaN have one without tokens.
struct RowSpan {
    int lo, hi, units;
    bool bad;
};
__device__ __forceinline__ RowSpan row_span(const AttendArgs& a, int n, int unit) {
    if (n < 0) return {0, 0, 0, false};
    if (n == 0 || n > a.most) return {0, 0, 1, n != 0};
    const int lo = a.window > 0 && n > a.window ? n - a.window : 0;
    return {lo, n, (n - 1) / unit - lo / unit + 1, false};
}

// A value equal in all lanes, in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Inclusive prefix sum over a wave's lanes.
__device__ __forceinline__ int wave_prefix(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // rows of 16: from 1, 2, 4, 8 lanes below
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row 0's sum to row 1, row 2's to row 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // the lower half's to the upper
    return v;
}

// Maximum over a wave's lanes, moved like the prefix sum.
__device__ __forceinline__ int wave_max(int v) {
    auto top = [](int a, int b) { return a > b ? a : b; };
    v = top(v, __builtin_amdgcn_update_dpp(v, v, 0x111, 0xF, 0xF, false));
    v = top(v, __builtin_amdgcn_update_dpp(v, v, 0x112, 0xF, 0xF, false));
    v = top(v, __builtin_amdgcn_update_dpp(v, v, 0x114, 0xF, 0xF, false));
    v = top(v, __builtin_amdgcn_update_dpp(v, v, 0x118, 0xF, 0xF, false));
    v = top(v, __builtin_amdgcn_update_dpp(v, v, 0x142, 0xA, 0xF, false));
    v = top(v, __builtin_amdgcn_update_dpp(v, v, 0x143, 0xC, 0xF, false));
    return __builtin_amdgcn_readlane(v, 63);
}

// n / d of numbers below 2^12, d > 0: half of one to spare makes it exact.  A
// few instructions, where the integer division has forty: code that runs once
// waits for its fetch (these quotients in place of divisions: 1 x 8192 tokens
// 12.75 -> 12.65 us, 1 x 131072 34.7 -> 34.4).
__device__ __forceinline__ int small_quotient(int n, int d) {
    return (int)(((float)n + 0.5f) * __builtin_amdgcn_rcpf((float)d));
}

// One workgroup's work: chunk `chunk` of `chunks` of a segment (row, kv head,
// 16 query heads), `size` units a chunk, and the number of the workgroup that
// has the segment's first.
struct Piece {
    int row, seg, length;
    int chunk, chunks, size, first;
};

// The piece of workgroup `w` of a launch that splits, counted from the lengths
// by every wave for itself, 64 rows at a time (up to 64 rows are read once).
// With U units in all segments, chunks have at least U / 2^target units, so
// there are at most 2^target + segments of them, and a segment has at most
// kAttendMaxParts.  With `other` for `target` only where there are at most
// 2^other: as many as fit side by side (of at most 64 rows).  False: there are
// fewer pieces.
__device__ __forceinline__ bool find_piece(const AttendArgs& a, int unit, int w, Piece& p) {
    int mine, units, longest = 0;
    uint32_t total = 0;   // fits: 256 rows of under 2^24 units
    auto load = [&](int r0) {
        const int r = r0 + (int)(threadIdx.x & 63);
        mine = r < a.rows ? gptr<int32_t>(a.lengths)[r] : -1;
        units = row_span(a, mine, unit).units;
    };
    // (backwards: the first 64 are there when the second pass starts)
    for (int r0 = (a.rows - 1) & ~63; r0 >= 0; r0 -= 64) {
        load(r0);
        total += (uint32_t)__builtin_amdgcn_readlane(wave_prefix(units), 63);
        const int most = wave_max(units);
        longest = longest > most ? longest : most;
    }
    const uint64_t all = (uint64_t)total * a.head_tiles.d;
    const int least = (longest + kAttendMaxParts - 1) / kAttendMaxParts;
    auto size_for = [&](int target) {
        const int even = (int)((all + (1u << target) - 1) >> target);
        return even > least ? even : least;
    };
    int size = longest > 0 ? longest : 1;
    int limit = 0, k = 0, most_k = 0;   // pieces that may come out (0: any), the size's twelfths above `size`, and how many
    if (longest > a.whole_units) {
        size = size_for(a.target);
        if (a.other) {
            const int lone = size_for(a.other);
            if (lone >= a.other_size && (float)total >= (float)longest * a.other_rows) {
                size = lone;
                limit = a.other;
                most_k = a.slack;
            }
        }
    }
    int before = 0;   // pieces of earlier rows
    for (int r0 = 0;;) {
        int chunks, v, sum;
        for (;;) {
            p.size = size + (size * k + 6) / 12;
            // a row's chunks: n / p.size, at most 32, or 1 in whole rows
            const int n = units + p.size - 1;
            chunks = (int)((float)n * __builtin_amdgcn_rcpf((float)p.size));
            chunks -= chunks * p.size > n;
            chunks += (chunks + 1) * p.size <= n;
            v = wave_prefix(chunks) * (int)a.head_tiles.d;
            sum = __builtin_amdgcn_readlane(v, 63);
            if (limit == 0 || sum <= 1 << limit) break;
            if (++k > most_k) {   // up to `other`, then up to `target` if that is more, then as they come
                k = 0;
                most_k = 6;
                size = size_for(a.target);
                limit = limit < a.target ? a.target : 0;
            }
        }
        if (w < before + sum) {
            const int at = __builtin_popcountll(__builtin_amdgcn_ballot_w64(before + v <= w));   // rows that end at or before w
            p.row = r0 + at;
            p.length = __builtin_amdgcn_readlane(mine, at);
            p.chunks = __builtin_amdgcn_readlane(chunks, at);
            before += __builtin_amdgcn_readlane(v, at) - p.chunks * (int)a.head_tiles.d;
            p.seg = uniform(small_quotient(w - before, p.chunks));
            p.first = before + p.seg * p.chunks;
            p.chunk = w - p.first;
            return true;
        }
        before += sum;
        r0 += 64;
        if (r0 >= a.rows) return false;
        load(r0);
    }
}

// Partial results follow the counters, a slot for each workgroup: the group's
// rows of head_dim sums, then each row's reference and sum of weights.
constexpr size_t slot_floats(int heads, int D) { return (size_t)heads * (D + 2); }

// Workspace traffic between workgroups, which may run on XCDs with L2s of
// their own: agent-scope accesses only, which do not stop at an L2.  So a
// store that has completed is seen by every later load, and no cache has to
// be written back or invalidated.  (Release and acquire at the counters, which
// do that to a whole L2 for every part, took twice as long: 113 us against 55
// for 131072 tokens at 4 bits when it was measured.)
typedef float f2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void put(float* p, f2 v) {
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f2 get(const float* p) {
    return __builtin_bit_cast(f2, __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// Whether this workgroup is the last of `n` to arrive at a counter, which then
// reads zero again.  What the workgroups put before is there for the last.
__device__ __forceinline__ bool last_of(uint32_t* counter, uint32_t n, bool* flag) {
    // each thread's stores have completed (a workgroup barrier does not wait for them), then one count.  To the compiler
    // the wait touches no memory: the empty clobber in front of it keeps the stores there.
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((0 & 15) | ((0 >> 4) << 14) | (7 << 4) | (15 << 8));   // vmcnt(0)
    __syncthreads();
    if (threadIdx.x == 0) {
        *flag = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
        if (*flag) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return *flag;
}

// Four channels of one head, summed: the sums and the sum of weights against
// the reference `top`.
struct Joined {
    f4 o;
    float top, sum;
};

// One output in fp16.  The weights' roundings to fp16 can push an average of
// values near 65504 past it: a finite one stays finite.
__device__ __forceinline__ uint32_t output_bits(float x) {
    const float kept = __builtin_amdgcn_fmed3f(x, -65504.0f, 65504.0f);
    return (uint32_t)f32_to_f16_bits(__builtin_fabsf(x) < __builtin_inff() ? kept : x);
}

// out and lse of four channels.
__device__ __forceinline__ void finish(const AttendArgs& a, int row, int head, int d, const Joined& j, bool empty) {
    const float inv = empty ? 0.0f : __builtin_amdgcn_rcpf(j.sum);
    u2v w;
    w[0] = output_bits(j.o[0] * inv) | (output_bits(j.o[1] * inv) << 16);
    w[1] = output_bits(j.o[2] * inv) | (output_bits(j.o[3] * inv) << 16);
    *gptr_w<u2v>(a.out + (int64_t)row * a.out_row + (int64_t)head * a.out_head + d) = w;
    if (d == 0 && a.lse)
        gptr_w<float>(a.lse)[(int64_t)row * a.q_heads + head] =
            empty ? -__builtin_inff() : (j.top + __builtin_amdgcn_logf(j.sum)) * kLn2;
}

// Slots first, first + step, .. below n of head h, channels d .. d + 3, joined
// in that order.
template <int D>
__device__ __forceinline__ Joined join_parts(const float* slots, size_t floats, int first, int step, int n, int hp, int h, int d) {
    Joined j = {{0, 0, 0, 0}, -3e38f, 0.0f};
    for (int i0 = first; i0 < n; i0 += step * kJoinBatch) {
        f2 rl[kJoinBatch], x[kJoinBatch], y[kJoinBatch];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            const float* p = slots + (size_t)(i0 + i * step < n ? i0 + i * step : i0) * floats;
            rl[i] = get(p + (size_t)hp * D + 2 * h);
            x[i] = get(p + (size_t)h * D + d);
            y[i] = get(p + (size_t)h * D + d + 2);
        }
        float top = j.top;
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) top = __builtin_fmaxf(top, rl[i][0]);
        const float keep = __builtin_amdgcn_exp2f(j.top - top);
        j.sum *= keep;
        j.o *= keep;
        j.top = top;
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            if (i0 + i * step < n) {
                const float f = __builtin_amdgcn_exp2f(rl[i][0] - top);
                j.sum += rl[i][1] * f;
                j.o += f4{x[i][0], x[i][1], y[i][0], y[i][1]} * f;
            }
        }
    }
    return j;
}

// Each tile is read once: non-temporal loads (32 x 4000 tokens in 16 bits 89.2
// us, with ordinary ones 96.1; 16 x 8192 in 8 bits 52.8 and 57.6).  A cache that
// still lies in the 256 MB last-level cache would come faster with ordinary ones
// (76 MB over and over 22.8 and 21.3), but between two steps of a sequence the
// other layers' caches and weights pass through.
constexpr int kStreamed = 2;

// Reads go through one buffer descriptor a tile: its address in scalar
// registers, a lane's place as a 32-bit offset from a compile-time start.
template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t* dst, __amdgpu_buffer_rsrc_t tile, int at, int start) {
    if constexpr (WORDS >= 4) {
        const u4v v = __builtin_amdgcn_raw_buffer_load_b128(tile, at, start, kStreamed);
        dst[0] = v[0]; dst[1] = v[1]; dst[2] = v[2]; dst[3] = v[3];
        load_words<WORDS - 4>(dst + 4, tile, at, start + 16);
    } else if constexpr (WORDS == 3) {
        typedef uint32_t u3v __attribute__((ext_vector_type(3)));
        const u3v v = __builtin_amdgcn_raw_buffer_load_b96(tile, at, start, kStreamed);
        dst[0] = v[0]; dst[1] = v[1]; dst[2] = v[2];
    } else if constexpr (WORDS == 2) {
        const u2v v = __builtin_amdgcn_raw_buffer_load_b64(tile, at, start, kStreamed);
        dst[0] = v[0]; dst[1] = v[1];
    } else if constexpr (WORDS == 1) {
        dst[0] = __builtin_amdgcn_raw_buffer_load_b32(tile, at, start, kStreamed);
    }
}

// A lane's share of the codes of a tile's keys or values, from byte `start` of it.
template <int D, int B> struct RawPart {
    static constexpr int WORDS = D / kCacheGroup * B / 4;
    uint32_t w[WORDS];
};

template <int D, int B>
__device__ __forceinline__ void load_codes(RawPart<D, B>& r, __amdgpu_buffer_rsrc_t tile, int start, int lane) {
    using P = CachePart<D, B>;
    static_for<0, P::CHUNKS>([&](auto jc) {
        constexpr int j = jc, n = (P::G - j * P::GPC < P::GPC ? P::G - j * P::GPC : P::GPC) * B / 4;
        load_words<n>(r.w + 4 * j, tile, lane * (4 * n), start + 1024 * j);
    });
}

// A lane's share of a tile's keys or values, as loaded: codes, and the scales
// of its token (keys) or of [G][its 4 tokens] (values).
template <int D, int B> struct RawKeys {
    RawPart<D, B> k;
    uint32_t s[(D / kCacheGroup + 1) / 2];
};
template <int D, int B> struct RawValues {
    RawPart<D, B> v;
    uint32_t s[2 * (D / kCacheGroup)];
};

template <int D, int B>
__device__ __forceinline__ void load_keys(RawKeys<D, B>& r, __amdgpu_buffer_rsrc_t tile, int lane) {
    constexpr int G = D / kCacheGroup, S = CachePart<D, B>::CODES;
    load_codes<D, B>(r.k, tile, 0, lane);
    if constexpr (B < 16) {
        const int at = (lane & 15) * (2 * G);
        if constexpr (G % 2) {   // a token's scales start at an even half: by halves
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(tile, at, S + 2 * g, kStreamed);
                r.s[g / 2] = g % 2 ? r.s[g / 2] | (v << 16) : v;
            }
        } else {
            load_words<G / 2>(r.s, tile, at, S);
        }
    }
}

template <int D, int KB, int B>
__device__ __forceinline__ void load_values(RawValues<D, B>& r, __amdgpu_buffer_rsrc_t tile, int lane) {
    constexpr int G = D / kCacheGroup, V = CachePart<D, KB>::BYTES;
    load_codes<D, B>(r.v, tile, V, lane);
    if constexpr (B < 16) load_words<2 * G>(r.s, tile, (lane >> 4) * (8 * G), V + CachePart<D, B>::CODES);
}

// Key operand of group g: channels 32 g + 8 q + (0..7) of the lane's token.
template <int D, int KB>
__device__ __forceinline__ h8 key_operand(const RawKeys<D, KB>& r, int g, const Nibbles& nib) {
    u4v o;
    if constexpr (KB == 16) {
        o = u4v{r.k.w[4 * g], r.k.w[4 * g + 1], r.k.w[4 * g + 2], r.k.w[4 * g + 3]};
    } else {
        const h2 both = as_h2(r.s[g / 2]);
        const h2 s = g % 2 ? __builtin_shufflevector(both, both, 1, 1) : __builtin_shufflevector(both, both, 0, 0);
        if constexpr (KB == 4) {
            const uint32_t w = r.k.w[g];
            static_for<0, 4>([&](auto e) { o[e.value] = __builtin_bit_cast(uint32_t, nib.pair<e.value>(w) * s); });
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = r.k.w[2 * g + e / 2];
                const uint32_t x = __builtin_amdgcn_perm(w, 0x64006400u, e % 2 ? 0x01070106u : 0x01050104u);
                o[e] = __builtin_bit_cast(uint32_t, (as_h2(x) - as_h2(kBiasedZero<8>)) * s);
            }
        }
    }
    return __builtin_bit_cast(h8, o);
}

// Value operand words of group g, half h, of one tile: the lane's four tokens
// of channel 32 g + 16 h + c (two words).
template <int D, int VB>
__device__ __forceinline__ u2v value_words(const RawValues<D, VB>& r, int g, int h, const Nibbles& nib) {
    if constexpr (VB == 16) {
        return u2v{r.v.w[4 * g + 2 * h], r.v.w[4 * g + 2 * h + 1]};
    } else if constexpr (VB == 4) {
        const uint32_t w = r.v.w[g];
        const h2 a = h ? nib.pair<1>(w) : nib.pair<0>(w), b = h ? nib.pair<3>(w) : nib.pair<2>(w);
        return u2v{__builtin_bit_cast(uint32_t, a * as_h2(r.s[2 * g])), __builtin_bit_cast(uint32_t, b * as_h2(r.s[2 * g + 1]))};
    } else {
        const uint32_t w = r.v.w[2 * g + h];
        return u2v{scaled(__builtin_amdgcn_perm(w, 0x64006400u, 0x01050104u), kBiasedZero<8>, r.s[2 * g]),
                   scaled(__builtin_amdgcn_perm(w, 0x64006400u, 0x01070106u), kBiasedZero<8>, r.s[2 * g + 1])};
    }
}

// Clears what the tokens of a tile outside [lo, hi) contribute to the second
// product (weights of 0 would still turn a NaN or infinity there into NaN):
// their scales, or in 16 bits their values.  t0: the lane's first token.
template <int D, int VB>
__device__ __forceinline__ void clear_values(RawValues<D, VB>& r, int t0, int lo, int hi) {
    constexpr int G = D / kCacheGroup;
    uint32_t m[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = t0 + 2 * i;
        m[i] = (t >= lo && t < hi ? 0xFFFFu : 0u) | (t + 1 >= lo && t + 1 < hi ? 0xFFFF0000u : 0u);
    }
    if constexpr (VB == 16) {
#pragma unroll
        for (int i = 0; i < RawPart<D, VB>::WORDS; ++i) r.v.w[i] &= m[i % 2];
    } else {
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) r.s[i] &= m[i % 2];
    }
}

// Attention of one wave over its tokens: online softmax with the running
// reference r (log2 domain) of each head (column lane % 16), the lane's share
// l of the weights' sum, and the output sums o.  Scores are computed
// transposed (rows: tokens, columns: heads), so the accumulator registers of
// two tiles are, after the exponential, the lane's operand of the second
// product as they stand: lane (q, head) holds tokens 4 q .. 4 q + 3 of each.
// That operand is fp16, as the values are: a weight is off by 2^-11 of itself at
// most, its sum l adds it unrounded.  Of the outputs' norm the error against 64
// bits is 2.4e-4 to 2.9e-4, with weights of 32 bits 2.1e-4, the rounding of the
// outputs.  Weights of 22 bits, in two operands, would take the second product
// twice.
template <int D, int KB, int VB> struct AttendWave {
    static constexpr int G = D / kCacheGroup;
    Nibbles nib;
    h8 q[G];
    f4 o[2 * G];
    float r, l;
    float limit;   // a score that passes r by more moves r; below any score until r is set

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) o[i] = f4{0, 0, 0, 0};
        r = l = 0.0f;
        limit = -3e38f;
    }
    __device__ __forceinline__ float reference() const { return limit < 0.0f ? -3e38f : r; }

    // The first half of a step: weights of the 32 tokens of two tiles, one after
    // the other.  ta: the lane's first token; partial: some lie outside [lo, hi).
    __device__ __forceinline__ h8 weights(const RawKeys<D, KB>& a, const RawKeys<D, KB>& b, float c, bool partial,
                                          int ta, int lo, int hi) {
        f4 sa = {0, 0, 0, 0}, sb = {0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < G; ++g) {
            sa = __builtin_amdgcn_mfma_f32_16x16x32_f16(key_operand(a, g, nib), q[g], sa, 0, 0, 0);
            sb = __builtin_amdgcn_mfma_f32_16x16x32_f16(key_operand(b, g, nib), q[g], sb, 0, 0, 0);
        }
        float t[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = __builtin_fmaf(sa[i], c, -r);
            t[4 + i] = __builtin_fmaf(sb[i], c, -r);
        }
        if (partial) {
            // token - lo, against the span's length: made here from a value the
            // compiler does not see through, so that steps inside the span pay nothing
            uint32_t at = (uint32_t)(ta - lo);
            asm volatile("" : "+v"(at));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (at + (uint32_t)i >= (uint32_t)(hi - lo)) t[i] = -__builtin_inff();
                if (at + (uint32_t)(16 + i) >= (uint32_t)(hi - lo)) t[4 + i] = -__builtin_inff();
            }
        }
        float m = __builtin_fmaxf(__builtin_fmaxf(__builtin_fmaxf(t[0], t[1]), __builtin_fmaxf(t[2], t[3])),
                                  __builtin_fmaxf(__builtin_fmaxf(t[4], t[5]), __builtin_fmaxf(t[6], t[7])));
        // The reference starts 2^7 below the largest weight seen and moves only
        // when a weight would pass 2^15: fp16 weights stay finite, and one is
        // lost to underflow only below 2^-31 of the largest.
        if (__builtin_amdgcn_ballot_w64(m > limit)) {
            m = __builtin_fmaxf(m, __shfl_xor(m, 16));
            m = __builtin_fmaxf(m, __shfl_xor(m, 32));
            const bool up = m > limit;
            const float by = up ? m - 7.0f : 0.0f;
            const float f = !up ? 1.0f : limit < 0.0f ? 0.0f : __builtin_amdgcn_exp2f(-by);   // nothing is summed before r is set
            if (up) limit = 15.0f;
            r += by;
            l *= f;
#pragma unroll
            for (int i = 0; i < 2 * G; ++i) o[i] *= f;
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] -= by;
        }
        h8 p;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = __builtin_amdgcn_exp2f(t[i]);
            l += e;
            p[i] = (_Float16)e;
        }
        return p;
    }

    // The second half: their values' weighted sums.
    __device__ __forceinline__ void sums(const RawValues<D, VB>& a, const RawValues<D, VB>& b, h8 p) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u2v x = value_words(a, g, h, nib), y = value_words(b, g, h, nib);
                const u4v w = {x[0], x[1], y[0], y[1]};
                o[2 * g + h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, w), p, o[2 * g + h], 0, 0, 0);
            }
    }
};

// Attention over the cache: a workgroup of NW waves takes one chunk of a
// segment, a unit of 32 NW tokens a step, each wave on 32 of them with a
// softmax of its own; the waves join in LDS, and the last workgroup of a
// segment to finish joins the parts of all, through the workspace.
//
// Bound by the cache's bytes where there are many (32 x 16384 tokens at 4 bits:
// 605 MB in 107 us, 5.7 TB/s; with the codes used as they are, two instructions in
// place of the decoding's 200 of a step's 240, 104; 32 x 4000 in 16 bits: 525 MB in
// 81 us, 6.5 TB/s of a plain read's 7.0), and by the chain of length, page number, first
// tile and join where there are few (100 tokens 5.5 us, 2048 in parts 9).
template <int D, int KB, int VB, int NW>
__global__ __launch_bounds__(64 * NW, (attend_waves_per_simd(D, KB, VB))) void attend_kernel(AttendArgs a) {
    using PK = CachePart<D, KB>;
    using PV = CachePart<D, VB>;
    constexpr int G = D / kCacheGroup, TILE = PK::BYTES + PV::BYTES, THREADS = 64 * NW, UNIT = 32 * NW;
    constexpr int PITCH = D + 4;   // heads' rows start four banks apart: 16 lanes store their head's sums side by side
    __shared__ __attribute__((aligned(16))) float part_o[NW][16][PITCH];
    __shared__ float part_r[NW][16], part_l[NW][16], part_f[NW][16];
    __shared__ bool last;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int quad = lane >> 4, col = lane & 15;

    Piece p;
    if (a.target == 0) {
        p.row = (int)a.head_tiles.divide(blockIdx.x);
        p.seg = (int)(blockIdx.x - (uint32_t)p.row * a.head_tiles.d);
        p.length = uniform(gptr<int32_t>(a.lengths)[p.row]);
        p.chunk = 0;
        p.chunks = 1;
        p.size = 0x7FFFFFFF;
        p.first = 0;
    } else if (!find_piece(a, UNIT, (int)blockIdx.x, p)) {
        return;
    }
    const RowSpan span = row_span(a, p.length, UNIT);
    if (span.units == 0) return;   // a padding row
    const int kvh = (int)a.group_tiles.divide((uint32_t)p.seg), hs = (p.seg - kvh * (int)a.group_tiles.d) * 16;
    const int h0 = kvh * a.group + hs, heads = a.group - hs < 16 ? a.group - hs : 16;
    AttendWave<D, KB, VB> W;
    W.nib.init();
    W.reset();
    // Query operand: channels 32 g + 8 q + (0..7) of head h0 + col.
    const uint16_t* qsrc = a.q + (int64_t)p.row * a.q_row + (int64_t)(h0 + (col < heads ? col : 0)) * a.q_head + 8 * quad;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        u4v w = *gptr<u4v>(qsrc + g * kCacheGroup);
        w &= col < heads ? 0xFFFFFFFFu : 0u;
        W.q[g] = __builtin_bit_cast(h8, w);
    }
    // The wave's steps: those of the chunk's units that hold a token of the span.
    const int first_unit = span.lo / UNIT, my = 32 * wave;
    int i0 = p.chunk * p.size, i1 = p.chunk + 1 < p.chunks ? i0 + p.size : span.units;
    {
        const int lo_steps = (span.lo - my - 32 + UNIT) / UNIT - first_unit;      // first with a token >= lo
        const int hi_steps = (span.hi - my + UNIT - 1) / UNIT - first_unit;       // past the last with one < hi
        i0 = i0 > lo_steps ? i0 : lo_steps;
        i1 = i1 < hi_steps ? i1 : hi_steps;
    }
    bool bad = span.bad;
    const int32_t* pages = a.t.pages + (int64_t)p.row * a.t.stride;
    // Lane j holds the numbers, among the cache's tiles, of the two tiles of
    // step c0 + j, 64 steps at a time: one look at the page table per 64 steps.
    const uint32_t all_tiles = a.c.tiles * a.c.kv_heads, head_tile = (uint32_t)kvh * a.c.tiles;
    uint32_t tile_a = 0, tile_b = 0;
    int c0 = 0;
    auto look_up = [&](int from) {
        c0 = from;
        const int i = from + lane;
        const int token = (first_unit + i) * UNIT + my;
        const bool live = i < i1;
        const bool ina = live && token + 16 > span.lo, inb = live && token + 16 < span.hi;
        auto number = [&](bool in, int tok, bool& odd) -> uint32_t {
            const uint32_t tile = (uint32_t)tok / kCacheTile, pi = a.page_tiles.divide(tile);
            uint32_t page = in ? (uint32_t)gptr<int32_t>(pages)[pi] : 0u;
            odd = page >= a.c.n_pages;
            if (odd) page = 0;
            return page * all_tiles + head_tile + (tile - pi * a.c.tiles);
        };
        bool odd_a, odd_b;
        tile_a = number(ina, token, odd_a);
        tile_b = number(inb, token + 16, odd_b);
        if (!ina) tile_a = tile_b;   // tiles without a token of the span are not read
        if (!inb) tile_b = tile_a;
        bad |= __builtin_amdgcn_ballot_w64(odd_a || odd_b) != 0;
    };
    auto tile_at = [&](uint32_t number, int i) {
        const uint32_t n = (uint32_t)__builtin_amdgcn_readlane((int)number, i - c0);
        return buffer_rsrc(a.c.pages + (uint64_t)n * TILE, (uint32_t)TILE);
    };
    // A wave's priority falls as its steps run out, at a half, a quarter and an
    // eighth of a chunk: of two waves on a SIMD the older one would be served
    // first and end when the younger still has a fifth to go, with nothing
    // beside it to hide its waits (131072 tokens at 4 bits 35.4 us, without it
    // 37.0; 64 ragged rows of up to 4096 41.2 and 45.2).  In 16 bits, where the
    // memory alone sets the pace, it gains nothing (53.6 and 52.9).
    constexpr bool kPaced = KB < 16;
    // Keys and values of one step each in registers: a step's keys are
    // asked for once the keys before are used up, under the second product,
    // and its values under the next step's first.  Past the end the last
    // step is loaded again, so that every wait knows what is in flight.
    if (i0 < i1) {
        RawKeys<D, KB> ka, kb;
        RawValues<D, VB> va, vb;
        look_up(i0);
        __amdgpu_buffer_rsrc_t pa = tile_at(tile_a, i0), pb = tile_at(tile_b, i0);
        load_keys(ka, pa, lane);
        load_keys(kb, pb, lane);
        load_values<D, KB>(va, pa, lane);
        load_values<D, KB>(vb, pb, lane);
        if constexpr (kPaced) __builtin_amdgcn_s_setprio(3);
        const int chunk_steps = p.size < span.units ? p.size : span.units;
        int pace_mark = chunk_steps / 2, pace = 3;
        for (int i = i0; i < i1; ++i) {
            if (kPaced && i1 - i <= pace_mark) {
                pace_mark /= 2;
                if (--pace == 2) __builtin_amdgcn_s_setprio(2);
                else if (pace == 1) __builtin_amdgcn_s_setprio(1);
                else __builtin_amdgcn_s_setprio(0);
            }
            const int next = i + 1 < i1 ? i + 1 : i;
            if (next - c0 >= 64) look_up(next);
            pa = tile_at(tile_a, next);
            pb = tile_at(tile_b, next);
            const int token = (first_unit + i) * UNIT + my;
            const bool partial = token < span.lo || token + 32 > span.hi;
            const h8 weights = W.weights(ka, kb, a.scale, partial, token + 4 * quad, span.lo, span.hi);
            __builtin_amdgcn_sched_barrier(0);   // not before the keys' registers are free
            load_keys(ka, pa, lane);
            load_keys(kb, pb, lane);
            if (partial) {
                clear_values(va, token + 4 * quad, span.lo, span.hi);
                clear_values(vb, token + 16 + 4 * quad, span.lo, span.hi);
            }
            W.sums(va, vb, weights);
            __builtin_amdgcn_sched_barrier(0);
            load_values<D, KB>(va, pa, lane);
            load_values<D, KB>(vb, pb, lane);
        }
    }
    // Join the waves.  (The thread's index through a register the compiler
    // does not see through: addresses made here stay out of the loop above.)
    int id = tid;
    asm volatile("" : "+v"(id));
    {
        const int quad = (id & 63) >> 4, col = id & 15;
        float l = W.l;
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (bad) l = __builtin_nanf("");
        if (quad == 0) {
            part_r[wave][col] = W.reference();
            part_l[wave][col] = l;
        }
        __syncthreads();
        float ref = part_r[0][col];
#pragma unroll
        for (int w = 1; w < NW; ++w) ref = __builtin_fmaxf(ref, part_r[w][col]);
        const float f = __builtin_amdgcn_exp2f(W.reference() - ref);
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) *reinterpret_cast<f4*>(&part_o[wave][col][16 * i + 4 * quad]) = W.o[i] * f;
        if (quad == 0) part_f[wave][col] = f;
        __syncthreads();
    }
    const int hp = a.group < 16 ? a.group : 16, items = heads * (D / 4);   // an item: four channels of a head
    const size_t floats = slot_floats(hp, D);
    float* slots = a.ws + kCounterBytes / sizeof(float);
    for (int i = id; i < items; i += THREADS) {
        const int h = i / (D / 4), d = i % (D / 4) * 4;
        Joined j = {{0, 0, 0, 0}, part_r[0][h], 0.0f};
#pragma unroll
        for (int w = 1; w < NW; ++w) j.top = __builtin_fmaxf(j.top, part_r[w][h]);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            j.sum += part_l[w][h] * part_f[w][h];
            j.o += *reinterpret_cast<const f4*>(&part_o[w][h][d]);
        }
        if (p.chunks == 1) {
            finish(a, p.row, h0 + h, d, j, span.hi == 0 && !span.bad);
        } else {
            float* slot = slots + (size_t)blockIdx.x * floats;
            put(slot + (size_t)h * D + d, f2{j.o[0], j.o[1]});
            put(slot + (size_t)h * D + d + 2, f2{j.o[2], j.o[3]});
            if (d == 0) put(slot + (size_t)hp * D + 2 * h, f2{j.top, j.sum});
        }
    }
    if (p.chunks == 1 || !last_of(reinterpret_cast<uint32_t*>(a.ws) + p.first, (uint32_t)p.chunks, &last)) return;
    // The last to finish joins the parts, in order: threads by items, and where
    // there are threads left over several of them on one item's parts.
    const float* parts = slots + (size_t)p.first * floats;
    const int ways = uniform(small_quotient(THREADS, items));   // 0: more items than threads
    if (ways <= 1) {
        for (int i = id; i < items; i += THREADS) {
            const int h = i / (D / 4), d = i % (D / 4) * 4;
            finish(a, p.row, h0 + h, d, join_parts<D>(parts, floats, 0, 1, p.chunks, hp, h, d), false);
        }
        return;
    }
    f4* way_o = reinterpret_cast<f4*>(&part_o[0][0][0]);                     // [THREADS]
    f2* way_rl = reinterpret_cast<f2*>(&part_o[0][0][0]) + 2 * THREADS;      // [THREADS]
    const int way = small_quotient(id, items), i = id - way * items, h = i / (D / 4), d = i % (D / 4) * 4;
    Joined j = {{0, 0, 0, 0}, -3e38f, 0.0f};
    if (way < ways) j = join_parts<D>(parts, floats, way, ways, p.chunks, hp, h, d);
    way_o[id] = j.o;
    way_rl[id] = f2{j.top, j.sum};
    __syncthreads();
    if (way != 0) return;
    for (int w = 1; w < ways; ++w) {
        const f2 rl = way_rl[w * items + i];
        const float top = __builtin_fmaxf(j.top, rl[0]);
        const float f = __builtin_amdgcn_exp2f(j.top - top), g = __builtin_amdgcn_exp2f(rl[0] - top);
        j.o = j.o * f + way_o[w * items + i] * g;
        j.sum = j.sum * f + rl[1] * g;
        j.top = top;
    }
    finish(a, p.row, h0 + h, d, j, false);
}

}  // namespace exq

// =================================================================== host

using namespace exq;

namespace {

bool cache_aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

exq_status check_geometry(int page_size, int kv_heads, int head_dim, int k_bits, int v_bits) {
    if (page_size < 16 || page_size > 65536 || page_size % 16)
        return fail(EXQ_ERR_INVALID_ARG, "page_size=%d is not a multiple of 16 in 16..65536", page_size);
    if (kv_heads < 1 || kv_heads > 65535) return fail(EXQ_ERR_INVALID_ARG, "kv_heads=%d outside 1..65535", kv_heads);
    if (head_dim < 32 || head_dim % 32) return fail(EXQ_ERR_INVALID_ARG, "head_dim=%d is not a positive multiple of 32", head_dim);
    if (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 256)
        return fail(EXQ_ERR_UNSUPPORTED, "head_dim=%d (only 64, 96, 128 and 256)", head_dim);
    const bool ks = k_bits == 4 || k_bits == 8, vs = v_bits == 4 || v_bits == 8;
    if (!((ks && vs) || (k_bits == 16 && v_bits == 16)))
        return fail(EXQ_ERR_UNSUPPORTED, "k_bits=%d v_bits=%d (each 4 or 8, or both 16)", k_bits, v_bits);
    return EXQ_OK;
}

CacheDev cache_dev(const exq_cache* c) {
    return CacheDev{c->pages, (int64_t)c->page_bytes, (uint32_t)c->n_pages, (uint32_t)c->page_size, (uint32_t)c->kv_heads,
                    (uint32_t)(c->page_size / kCacheTile)};
}

// An fp16 operand of (rows, heads, head_dim) with element strides.
struct Operand {
    const char* name;
    const void* p;
    int64_t row, head;
    int rows, heads, dim;
};

constexpr int64_t kMaxStride = (int64_t)1 << 30;   // elements: with 2^31 rows and heads extents stay inside 64 bits

exq_status check_operand(const Operand& x) {
    if (!x.p) return fail(EXQ_ERR_INVALID_ARG, "%s is NULL", x.name);
    if (!cache_aligned(x.p, 16)) return fail(EXQ_ERR_INVALID_ARG, "%s must be 16-byte aligned", x.name);
    if (x.row < 0 || x.head < 0 || x.row % 8 || x.head % 8 || x.row > kMaxStride || x.head > kMaxStride)
        return fail(EXQ_ERR_INVALID_ARG, "%s: strides (%lld, %lld) must be multiples of 8 in 0..2^30", x.name,
                    (long long)x.row, (long long)x.head);
    return EXQ_OK;
}

size_t extent(const Operand& x) {   // bytes from its first element to past its last
    return 2 * ((size_t)(x.rows - 1) * (size_t)x.row + (size_t)(x.heads - 1) * (size_t)x.head + (size_t)x.dim);
}

bool ranges_meet(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

// Whether no element of x is written twice.
bool distinct(const Operand& x) {
    const int64_t rows = x.rows, heads = x.heads, dim = x.dim;
    const bool rows_outer = (heads == 1 || x.head >= dim) && (rows == 1 || x.row >= (heads - 1) * x.head + dim);
    const bool heads_outer = (rows == 1 || x.row >= dim) && (heads == 1 || x.head >= (rows - 1) * x.row + dim);
    return rows_outer || heads_outer;
}

// Whether two operands may share memory.  Slices of one buffer's rows (equal
// row strides, disjoint within the row) do not, although their extents meet.
bool operands_meet(const Operand& a, const Operand& b) {
    if (!ranges_meet(a.p, extent(a), b.p, extent(b))) return false;
    if (a.row != b.row || a.row == 0) return true;
    const int64_t stride = 2 * a.row, na = 2 * ((a.heads - 1) * a.head + a.dim), nb = 2 * ((b.heads - 1) * b.head + b.dim);
    const int64_t diff = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
    const int64_t at = ((diff % stride) + stride) % stride;   // where b's rows start within a's stride
    return !(na <= at && at + nb <= stride);
}

exq_status check_table(const int32_t* table, int rows, int width, int64_t stride) {
    if (!table || !cache_aligned(table, 4)) return fail(EXQ_ERR_INVALID_ARG, "table is NULL or misaligned");
    if (rows < 1 || width < 1) return fail(EXQ_ERR_INVALID_ARG, "table of %d x %d", rows, width);
    if (stride < 0 || stride > kMaxStride || (rows > 1 && stride != 0 && stride < width))
        return fail(EXQ_ERR_INVALID_ARG, "table_stride=%lld", (long long)stride);
    return EXQ_OK;
}

// Bytes of a table from its first element to past its last.
size_t table_extent(int rows, int width, int64_t stride) {
    return 4 * ((size_t)(rows - 1) * (size_t)stride + (size_t)width);
}

// Calls f(IC<D>, IC<KB>, IC<VB>) for the cache's geometry.
template <class F>
void with_geometry(const exq_cache* c, F&& f) {
    auto bits = [&](auto d) {
        if (c->k_bits == 16) f(d, IC<16>{}, IC<16>{});
        else if (c->k_bits == 8 && c->v_bits == 8) f(d, IC<8>{}, IC<8>{});
        else if (c->k_bits == 8) f(d, IC<8>{}, IC<4>{});
        else if (c->v_bits == 8) f(d, IC<4>{}, IC<8>{});
        else f(d, IC<4>{}, IC<4>{});
    };
    switch (c->head_dim) {
        case 64: bits(IC<64>{}); break;
        case 96: bits(IC<96>{}); break;
        case 128: bits(IC<128>{}); break;
        default: bits(IC<256>{}); break;
    }
}

constexpr int64_t kMaxLaunchThreads = 0xFFFFFFFFll;

exq_status launched(const char* what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? EXQ_OK : fail(EXQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Waves of an append or read: a head of 16 rows each, and one block of rows
// more than there are, for blocks that start at the first row's tile.
int64_t rows_waves(const exq_cache* c, int rows) { return (((int64_t)rows + kCacheTile - 1) / kCacheTile + 1) * c->kv_heads; }
unsigned rows_workgroups(const exq_cache* c, int rows) {
    constexpr int per = kRowsThreads / 64;
    return (unsigned)((rows_waves(c, rows) + per - 1) / per);
}

exq_status check_rows_call(const exq_cache* c, const Operand& k, const Operand& v, int rows, const int32_t* table,
                           int table_rows, int table_width, int64_t table_stride, const int32_t* seqs,
                           const int32_t* positions) {
    if (rows < 0) return fail(EXQ_ERR_INVALID_ARG, "rows=%d", rows);
    if (table_rows < 0 || table_width < 0) return fail(EXQ_ERR_INVALID_ARG, "table of %d x %d", table_rows, table_width);
    if (rows == 0) return EXQ_OK;   // a step without rows: the tensors may be empty, their pointers NULL
    exq_status st;
    if ((st = check_table(table, table_rows, table_width, table_stride)) != EXQ_OK) return st;
    if ((st = check_operand(k)) != EXQ_OK || (st = check_operand(v)) != EXQ_OK) return st;
    if (!seqs || !positions || !cache_aligned(seqs, 4) || !cache_aligned(positions, 4))
        return fail(EXQ_ERR_INVALID_ARG, "seqs or positions is NULL or misaligned");
    const size_t bytes = (size_t)c->n_pages * c->page_bytes;
    if (ranges_meet(k.p, extent(k), c->pages, bytes) || ranges_meet(v.p, extent(v), c->pages, bytes))
        return fail(EXQ_ERR_INVALID_ARG, "k or v overlaps the cache's pages");
    if (rows_waves(c, rows) > kMaxLaunchThreads / 64 - 8)
        return fail(EXQ_ERR_UNSUPPORTED, "%d rows of %d heads in one call", rows, c->kv_heads);
    return EXQ_OK;
}

// Whether [p, p + n), which a rows call writes, meets the table, seqs or
// positions, which it reads.
bool meets_indices(const void* p, size_t n, int rows, const int32_t* table, int table_rows, int table_width,
                   int64_t table_stride, const int32_t* seqs, const int32_t* positions) {
    return ranges_meet(p, n, table, table_extent(table_rows, table_width, table_stride)) ||
           ranges_meet(p, n, seqs, 4 * (size_t)rows) || ranges_meet(p, n, positions, 4 * (size_t)rows);
}

// Tokens of all segments from which on attend_full geometries take a workgroup
// for every place the card has for one.  Measured on rows of 16384 tokens and 8
// heads, four workgroups a CU against one or two: head_dim 128, 8 rows 38 and 37
// us, 12 57.6 and 50.3, 16 60.0 and 58.8, 20 90.5 and 79.2, 24 92.2 and 101.3, 28
// 100 and 105, 32 104.7 and 107.2, 48 190 and 190; head_dim 64, 16 rows 37.7 and
// 43.0, 24 62 and 74.7, 32 63 and 76, 48 124.6 and 124.6, 64 115 and 137.5.  So
// the gain sets in at 3.1 million tokens of 128 channels and at 2.1 of 64 already;
// the limit is above both, and calls between them and it do without.
constexpr int64_t kFullTokens = (int64_t)1 << 22;

// Shape of an exq_attend launch.
struct AttendPlan {
    int head_tiles, wgs, waves;   // waves of a workgroup
    int target, whole_units;
    int other, other_size, slack;
    float other_rows;
    size_t ws_bytes;
};

exq_status plan_attend(const exq_cache* c, int rows, int q_heads, int table_width, AttendPlan* out) {
    if (rows < 0) return fail(EXQ_ERR_INVALID_ARG, "rows=%d", rows);
    if (q_heads < 1 || q_heads % c->kv_heads)
        return fail(EXQ_ERR_INVALID_ARG, "q_heads=%d is not a positive multiple of kv_heads=%d", q_heads, c->kv_heads);
    if (table_width < (rows > 0)) return fail(EXQ_ERR_INVALID_ARG, "table_width=%d", table_width);
    const int group = q_heads / c->kv_heads;
    const int64_t tiles = (int64_t)c->kv_heads * ((group + 15) / 16), segments = tiles * rows;
    if (segments > kMaxLaunchThreads / 256)
        return fail(EXQ_ERR_UNSUPPORTED, "%d rows of %d heads in one call", rows, q_heads);
    // Of the longest row there may be: the lengths are on the device.  The figures
    // below are of tables about as wide as the rows.  In one for 131072 tokens the
    // choices are those for long rows: 100 tokens take 5.4 us in place of 4.6, 2048
    // 11.0 in place of 8.8, 4 x 4096 13.0 in place of 11.6, 16 x 900 10.9 in place of
    // 10.1, 12 x 8192 33.8 in place of 30.0, 5 x 1999 of a window of 1023 in 8 bits
    // 11.3 in place of 8.4.
    const int64_t tokens = (int64_t)table_width * c->page_size;
    // Workgroups of 8 waves, one a CU, for few segments of long rows whose steps
    // are light: a segment has half as many parts to join (at 4 bits, 131072
    // tokens of 8 heads 35.4 us, with 4 waves 47.8; 4 x 16384 22.7 and 26.9; but
    // 4 x 4096 13.5 and 12.9; at 8 bits 4 x 16384 33.6 and 32.2).
    const bool eight = segments < 64 && tokens >= 16384 && attend_light(c->head_dim, c->k_bits, c->v_bits);
    out->waves = eight ? 8 : 4;
    out->head_tiles = (int)tiles;
    const int unit = 32 * out->waves;
    const int64_t units = (tokens - 1) / unit + 1;
    // Rows that are not worth splitting: joining their parts costs what 640
    // tokens cost where few workgroups run (one row of 800 tokens 10.9 us whole,
    // 9.1 split; 600 tokens 8.9 and 9.2), 1024 where a quarter of the card does (8
    // rows of 8 heads, 1000 tokens 11.6 whole, 12.6 split; 16 x 2000 22.1 and
    // 16.7), and 2048 where all of it does (32 x 2000 23.4 and 23.2).  Very many
    // are not split at all (kAttendMaxSegments): every workgroup would look
    // through all rows' lengths.
    out->whole_units = (segments >= kCus ? 2048 : segments >= 64 ? 1024 : 640) / unit;
    const bool split = units > out->whole_units && rows > 0 && segments <= kAttendMaxSegments && rows <= kAttendMaxRows;
    // With 64 segments or more, two workgroups a CU balance rows of different
    // lengths (at 4 bits 16 ragged rows of up to 8192 tokens 23.2 us, with one a
    // CU 30.8; equal rows of 4096 22.8 and 26.8); below that they only add parts
    // (4 x 4096 tokens 13.4, with one a CU 12.9).
    out->target = split ? (segments >= 64 ? kCusLog2 + 1 : kCusLog2) : 0;
    // Other numbers, where the lengths come out at no more than those with chunks
    // that are a little longer:
    // - heavy steps fill the memory's queues by themselves.  One workgroup a CU (16
    //   x 4096 tokens in 16 bits 47.9 us, with two 52.8; 24 x 4096 62.0 and 81.4; 16
    //   x 8192 ragged 43.5 and 49.3; head_dim 256, 20 x 4096 in 8 bits 40.0 and
    //   50.5), with chunks up to a third longer where a token has 384 bytes or more,
    //   else of the equal size only (16 x 8192 ragged in 8 bits 33.4, with two
    //   31.1); failing that exactly two, with chunks up to half longer (32 x 4000
    //   ragged in 8 bits 35.5 us, with what they come out at 39.5).  More segments
    //   than CUs make two of that kind anyway;
    // - light ones: exactly two if the rows are about equally long (12 x 8192 at 4
    //   bits 30.2 us, with what they come out at 33.8; 11 x 8192 in 4 and 8 bits
    //   34.6 and 39.5; ragged rows would lose, 32 x 16384 85.8 and 77.7);
    // - four, all that fit, for very long rows at 4 bits, whose decoding waits for
    //   loads (32 x 16384 105 us, with two 107; head_dim 64, 64 x 16384 115 and 137;
    //   but 16 x 16384 60.0 and 58.8, and head_dim 96, 32 x 16384 108.4 and 105.8).
    const bool heavy = !attend_light(c->head_dim, c->k_bits, c->v_bits);
    const bool full = attend_full(c->head_dim, c->k_bits, c->v_bits) && segments * tokens >= kFullTokens;
    // Below 64 segments one a CU is the aim already, and a few workgroups more
    // would double it for some: chunks up to a third longer if that makes them
    // fit (5 x 16384 tokens at 4 bits 27.2 us, without 35.2; 6 x 8192 in 16 bits
    // 38.9 and 51.6).  8 segments have 256 parts at most.
    const bool few = segments < 64;
    const bool whole_card = !few && full;
    out->other = !split || rows > 64 ? 0 : few ? (segments * kAttendMaxParts > kCus ? kCusLog2 : 0)
                 : whole_card ? kCusLog2 + 2 : segments > kCus ? 0 : heavy ? kCusLog2 : kCusLog2 + 1;
    out->slack = whole_card || (!few && heavy && row_bytes(c->head_dim, c->k_bits, c->v_bits) < 384) ? 0 : 4;
    out->other_size = whole_card ? (int)(kFullTokens / unit >> out->other) : 2;   // chunks of one unit fit as they are
    out->other_rows = few || heavy ? 0.0f : 0.875f * (float)rows;
    out->wgs = split ? (int)std::min<int64_t>(std::max<int64_t>((1 << out->target) + segments, out->other ? 1 << out->other : 0),
                                              segments * std::min<int64_t>(units, kAttendMaxParts))
                     : (int)segments;
    out->ws_bytes = split ? kCounterBytes + (size_t)out->wgs * sizeof(float) * slot_floats(std::min(group, 16), c->head_dim) : 0;
    return EXQ_OK;
}

}  // namespace

extern "C" {

size_t exq_cache_page_bytes(int page_size, int kv_heads, int head_dim, int k_bits, int v_bits) {
    if (check_geometry(page_size, kv_heads, head_dim, k_bits, v_bits) != EXQ_OK) return 0;
    return (size_t)page_size * kv_heads * row_bytes(head_dim, k_bits, v_bits);
}

exq_status exq_cache_create(void* pages, int64_t n_pages, int page_size, int kv_heads, int head_dim, int k_bits,
                            int v_bits, exq_cache_t* out) {
    if (!out) return fail(EXQ_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    const exq_status st = check_geometry(page_size, kv_heads, head_dim, k_bits, v_bits);
    if (st != EXQ_OK) return st;
    if (!pages || !cache_aligned(pages, 16)) return fail(EXQ_ERR_INVALID_ARG, "pages is NULL or not 16-byte aligned");
    if (n_pages < 1 || n_pages > 0x7FFFFFFFll)
        return fail(EXQ_ERR_INVALID_ARG, "n_pages=%lld outside 1..2^31-1", (long long)n_pages);
    if (n_pages * kv_heads > 0xFFFFFFFFll / (page_size / kCacheTile))   // tiles are numbered in 32 bits
        return fail(EXQ_ERR_UNSUPPORTED, "%lld pages of %d tokens and %d heads: over 2^32 tiles of 16 tokens",
                    (long long)n_pages, page_size, kv_heads);
    exq_cache* c = new (std::nothrow) exq_cache();
    if (!c) return fail(EXQ_ERR_OOM, "host allocation");
    *c = exq_cache{static_cast<uint8_t*>(pages), n_pages, page_size, kv_heads, head_dim, k_bits, v_bits,
                   exq_cache_page_bytes(page_size, kv_heads, head_dim, k_bits, v_bits)};
    *out = c;
    return EXQ_OK;
}

void exq_cache_destroy(exq_cache_t c) { delete c; }

exq_status exq_cache_append(exq_cache_t c, const void* k, int64_t k_row_stride, int64_t k_head_stride, const void* v,
                            int64_t v_row_stride, int64_t v_head_stride, int rows, const int32_t* table, int table_rows,
                            int table_width, int64_t table_stride, const int32_t* seqs, const int32_t* positions,
                            void* stream) {
    if (!c) return fail(EXQ_ERR_INVALID_ARG, "cache is NULL");
    const Operand ko{"k", k, k_row_stride, k_head_stride, rows, c->kv_heads, c->head_dim};
    const Operand vo{"v", v, v_row_stride, v_head_stride, rows, c->kv_heads, c->head_dim};
    const exq_status st =
        check_rows_call(c, ko, vo, rows, table, table_rows, table_width, table_stride, seqs, positions);
    if (st != EXQ_OK || rows == 0) return st;
    if (meets_indices(c->pages, (size_t)c->n_pages * c->page_bytes, rows, table, table_rows, table_width, table_stride, seqs, positions))
        return fail(EXQ_ERR_INVALID_ARG, "table, seqs or positions overlaps the cache's pages");
    const CacheDev d = cache_dev(c);
    const TableDev t{table, table_stride, (uint32_t)table_rows, (uint32_t)table_width};
    const dim3 grid(rows_workgroups(c, rows));
    with_geometry(c, [&](auto D, auto KB, auto VB) {
        hipLaunchKernelGGL((append_kernel<D.value, KB.value, VB.value>), grid, dim3(kRowsThreads), 0,
                           static_cast<hipStream_t>(stream), d, t, static_cast<const uint16_t*>(k), k_row_stride,
                           k_head_stride, static_cast<const uint16_t*>(v), v_row_stride, v_head_stride, rows, seqs, positions);
    });
    return launched("cache append launch");
}

exq_status exq_cache_read(exq_cache_t c, void* k, int64_t k_row_stride, int64_t k_head_stride, void* v,
                          int64_t v_row_stride, int64_t v_head_stride, int rows, const int32_t* table, int table_rows,
                          int table_width, int64_t table_stride, const int32_t* seqs, const int32_t* positions,
                          void* stream) {
    if (!c) return fail(EXQ_ERR_INVALID_ARG, "cache is NULL");
    const Operand ko{"k", k, k_row_stride, k_head_stride, rows, c->kv_heads, c->head_dim};
    const Operand vo{"v", v, v_row_stride, v_head_stride, rows, c->kv_heads, c->head_dim};
    const exq_status st =
        check_rows_call(c, ko, vo, rows, table, table_rows, table_width, table_stride, seqs, positions);
    if (st != EXQ_OK || rows == 0) return st;
    if (!distinct(ko) || !distinct(vo)) return fail(EXQ_ERR_INVALID_ARG, "rows or heads of k or v overlap themselves");
    if (operands_meet(ko, vo)) return fail(EXQ_ERR_INVALID_ARG, "k and v overlap");
    if (meets_indices(k, extent(ko), rows, table, table_rows, table_width, table_stride, seqs, positions) ||
        meets_indices(v, extent(vo), rows, table, table_rows, table_width, table_stride, seqs, positions))
        return fail(EXQ_ERR_INVALID_ARG, "k or v overlaps table, seqs or positions");
    const CacheDev d = cache_dev(c);
    const TableDev t{table, table_stride, (uint32_t)table_rows, (uint32_t)table_width};
    const dim3 grid(rows_workgroups(c, rows));
    with_geometry(c, [&](auto D, auto KB, auto VB) {
        hipLaunchKernelGGL((cache_read_kernel<D.value, KB.value, VB.value>), grid, dim3(kRowsThreads), 0,
                           static_cast<hipStream_t>(stream), d, t, static_cast<uint16_t*>(k), k_row_stride, k_head_stride,
                           static_cast<uint16_t*>(v), v_row_stride, v_head_stride, rows, seqs, positions);
    });
    return launched("cache read launch");
}

size_t exq_attend_workspace_bytes(exq_cache_t c, int rows, int q_heads, int table_width) {
    AttendPlan p;
    if (!c) {
        (void)fail(EXQ_ERR_INVALID_ARG, "cache is NULL");
        return 0;
    }
    return plan_attend(c, rows, q_heads, table_width, &p) == EXQ_OK ? p.ws_bytes : 0;
}

exq_status exq_attend(exq_cache_t c, const void* q, int64_t q_row_stride, int64_t q_head_stride, int rows, int q_heads,
                      const int32_t* table, int table_width, int64_t table_stride, const int32_t* lengths, float scale,
                      int window, void* out, int64_t out_row_stride, int64_t out_head_stride, float* lse,
                      void* workspace, size_t workspace_bytes, void* stream) {
    if (!c) return fail(EXQ_ERR_INVALID_ARG, "cache is NULL");
    AttendPlan p;
    exq_status st = plan_attend(c, rows, q_heads, table_width, &p);
    if (st != EXQ_OK) return st;
    if (!std::isfinite(scale * kLog2e)) return fail(EXQ_ERR_INVALID_ARG, "scale=%g is not finite or too large", (double)scale);
    if (window < 0) return fail(EXQ_ERR_INVALID_ARG, "window=%d", window);
    if (rows == 0) return EXQ_OK;
    if ((st = check_table(table, rows, table_width, table_stride)) != EXQ_OK) return st;
    const Operand qo{"q", q, q_row_stride, q_head_stride, rows, q_heads, c->head_dim};
    const Operand oo{"out", out, out_row_stride, out_head_stride, rows, q_heads, c->head_dim};
    if ((st = check_operand(qo)) != EXQ_OK || (st = check_operand(oo)) != EXQ_OK) return st;
    if (!lengths || !cache_aligned(lengths, 4) || !cache_aligned(lse, 4))
        return fail(EXQ_ERR_INVALID_ARG, "lengths is NULL, or lengths or lse misaligned");
    if (!distinct(oo)) return fail(EXQ_ERR_INVALID_ARG, "rows or heads of out overlap themselves");
    const size_t bytes = (size_t)c->n_pages * c->page_bytes;
    if (operands_meet(qo, oo) || ranges_meet(out, extent(oo), c->pages, bytes))
        return fail(EXQ_ERR_INVALID_ARG, "out overlaps q or the cache's pages");
    const size_t lse_bytes = lse ? 4 * (size_t)rows * q_heads : 0;
    if (lse && (ranges_meet(lse, lse_bytes, out, extent(oo)) || ranges_meet(lse, lse_bytes, q, extent(qo)) ||
                ranges_meet(lse, lse_bytes, c->pages, bytes)))
        return fail(EXQ_ERR_INVALID_ARG, "lse overlaps q, out or the cache's pages");
    const size_t table_bytes = table_extent(rows, table_width, table_stride), lengths_bytes = 4 * (size_t)rows;
    auto meets_read = [&](const void* x, size_t n) {   // of what every workgroup reads for itself
        return ranges_meet(x, n, table, table_bytes) || ranges_meet(x, n, lengths, lengths_bytes);
    };
    if (meets_read(out, extent(oo)) || (lse && meets_read(lse, lse_bytes)))
        return fail(EXQ_ERR_INVALID_ARG, "out or lse overlaps table or lengths");
    if (p.ws_bytes) {
        if (!workspace || !cache_aligned(workspace, 16) || workspace_bytes < p.ws_bytes)
            return fail(EXQ_ERR_INVALID_ARG, "workspace of %zu bytes: %zu 16-byte aligned ones are needed", workspace_bytes, p.ws_bytes);
        if (ranges_meet(workspace, p.ws_bytes, out, extent(oo)) || ranges_meet(workspace, p.ws_bytes, q, extent(qo)) ||
            ranges_meet(workspace, p.ws_bytes, c->pages, bytes) || (lse && ranges_meet(workspace, p.ws_bytes, lse, lse_bytes)) ||
            meets_read(workspace, p.ws_bytes))
            return fail(EXQ_ERR_INVALID_ARG, "workspace overlaps q, out, lse, table, lengths or the cache's pages");
    }
    AttendArgs a;
    a.c = cache_dev(c);
    a.t = TableDev{table, table_stride, (uint32_t)rows, (uint32_t)table_width};
    a.q = static_cast<const uint16_t*>(q);
    a.q_row = q_row_stride;
    a.q_head = q_head_stride;
    a.out = static_cast<uint16_t*>(out);
    a.out_row = out_row_stride;
    a.out_head = out_head_stride;
    a.lse = lse;
    a.lengths = lengths;
    a.ws = static_cast<float*>(workspace);
    a.scale = scale * kLog2e;
    a.window = window;
    a.most = (int)std::min<int64_t>(kMaxLength, (int64_t)table_width * c->page_size);
    a.rows = rows;
    a.q_heads = q_heads;
    a.group = q_heads / c->kv_heads;
    a.head_tiles = Divisor::of((uint32_t)p.head_tiles);
    a.group_tiles = Divisor::of((uint32_t)(a.group + 15) / 16);
    a.page_tiles = Divisor::of(a.c.tiles);
    a.target = p.target;
    a.other = p.other;
    a.other_size = p.other_size;
    a.other_rows = p.other_rows;
    a.slack = p.slack;
    a.whole_units = p.whole_units;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    with_geometry(c, [&](auto D, auto KB, auto VB) {
        auto launch = [&](auto NW) {
            hipLaunchKernelGGL((attend_kernel<D.value, KB.value, VB.value, NW.value>), dim3((unsigned)p.wgs), dim3(64 * NW.value), 0, s, a);
        };
        if constexpr (attend_light(D.value, KB.value, VB.value)) {
            if (p.waves == 8) {
                launch(IC<8>{});
                return;
            }
        }
        launch(IC<4>{});
    });
    return launched("attend launch");
}

}  // extern "C"
