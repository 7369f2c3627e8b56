// Pages of a key-value cache handed out to sequences and taken back on the GPU
// (exq_pages_extend, exq_pages_trim), with the sequence and position of every
// new row.  include/exq.h says what they compute.
//
// Both are a prefix sum over the sequences, of the pages that move and of the
// new rows, and then one look-up for every page and row: the sequence whose
// range holds it.  Nothing is ordered by atomics, so the same inputs give the
// same pages.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "exq_device_common.h"
#include "exq_internal.h"
#include "exq_operand.h"

namespace exq {

struct PagesArgs {
    int32_t* table;
    int64_t stride;
    int sequences, width, page_size;
    int32_t* lengths;
    const int32_t* change;   // extend: tokens to add; trim: tokens to keep
    int32_t* free_pages;
    int32_t* free_count;
    int n_pages;
    // extend only
    int32_t *seqs, *positions, *offsets, *served;
    int rows;
    // [sequences + 1] pages before each sequence's, [sequences] the first of its
    // columns, and the free list's count before the call
    int32_t *page_off, *first, *top;
};

constexpr int kPagesThreads = 1024;
constexpr int kPagesEach = 4;                                   // sequences of a thread in one pass
constexpr int kPagesChunk = kPagesThreads * kPagesEach;         // sequences of one pass

// Where the spreading half of a call finds the prefix sums: in LDS if one pass
// held them all, else in memory.
struct PagesView {
    const int32_t *rows_off, *page_off, *first;
    int sequences, top, pages, rows;
};

// The last s of [0, n) with off[s] <= x (off[0] = 0, ascending, x below off[n]):
// the one whose range [off[s], off[s + 1]) holds x.
template <class P> __device__ __forceinline__ int holder(P off, int n, int x) {
    int lo = 0, hi = n;   // off[lo] <= x < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Pages and rows first, first + step, .. of a call.
template <bool EXTEND>
__device__ __forceinline__ void pages_spread(const PagesArgs& a, const PagesView& v, int64_t first, int64_t step) {
    for (int64_t j = first; j < v.pages; j += step) {
        const int s = holder(v.page_off, v.sequences, (int)j);
        int32_t* entry = a.table + (int64_t)s * a.stride + (v.first[s] + ((int)j - v.page_off[s]));
        if (EXTEND) {
            *entry = a.free_pages[v.top - 1 - (int)j];
        } else {
            const int64_t to = (int64_t)v.top + v.pages - 1 - j;
            if (to < a.n_pages) a.free_pages[to] = *entry;
            *entry = -1;
        }
    }
    if (!EXTEND) return;
    for (int64_t r = first; r < a.rows; r += step) {
        int s = -1, position = 0;
        if (r < v.rows) {
            s = holder(v.rows_off, v.sequences, (int)r);
            // the sequence's new length, counted back from its last new row
            position = a.lengths[s] - (v.rows_off[s + 1] - (int)r);
        }
        a.seqs[r] = s;
        a.positions[r] = position;
    }
}

// Inclusive sums over a wave's lanes.
__device__ __forceinline__ int64_t wave_sums(int64_t x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    return x;
}

__device__ __forceinline__ int pages_of(int64_t tokens, int page_size) {
    return tokens <= 0 ? 0 : (int)((uint32_t)(tokens - 1) / (uint32_t)page_size) + 1;
}

// One workgroup looks through all sequences; with SPREAD it also does the rest.
template <bool EXTEND, bool SPREAD>
__global__ __launch_bounds__(kPagesThreads) void pages_scan_kernel(PagesArgs a) {
    __shared__ int32_t lds_rows[EXTEND && SPREAD ? kPagesChunk + 1 : 1];
    __shared__ int32_t lds_page[SPREAD ? kPagesChunk + 1 : 1], lds_first[SPREAD ? kPagesChunk : 1];
    __shared__ int64_t wave_total[2][kPagesThreads / 64];
    __shared__ int lds_stop;
    const int t = threadIdx.x, wave = t / 64, lane = t % 64, waves = blockDim.x / 64;
    const int chunk = blockDim.x * kPagesEach;
    const int64_t most = std::min<int64_t>((int64_t)a.width * a.page_size, 0x7FFFFFFF);
    const int top = min(max(*a.free_count, 0), a.n_pages);
    int64_t rows_before = 0, pages_before = 0;
    int stop = a.sequences;   // the first sequence that does not fit
    for (int base = 0; base < a.sequences; base += chunk) {
        int n[kPagesEach], add[kPagesEach], from[kPagesEach], need[kPagesEach];
        int64_t rows = 0, pages = 0;
        if (t == 0) lds_stop = a.sequences;
#pragma unroll
        for (int i = 0; i < kPagesEach; ++i) {
            const int s = base + t * kPagesEach + i;
            const bool in = s < a.sequences && stop == a.sequences;
            n[i] = in ? a.lengths[s] : -1;
            const int c = in ? a.change[s] : 0;
            add[i] = from[i] = need[i] = 0;
            if (EXTEND) {
                add[i] = n[i] < 0 ? 0 : max(c, 0);
                from[i] = pages_of(n[i], a.page_size);
                // what does not fit the table counts as more than there can be
                const int64_t end = (int64_t)n[i] + add[i];
                need[i] = add[i] == 0 ? 0 : end > most ? 0x7FFFFFFF : pages_of(end, a.page_size) - from[i];
            } else if (c >= 0 && c < n[i]) {
                add[i] = 1;   // the length changes
                const int64_t held = std::min<int64_t>(n[i], most);
                from[i] = pages_of(std::min<int64_t>(c, held), a.page_size);
                need[i] = pages_of(held, a.page_size) - from[i];
                n[i] = c;
            }
            if (EXTEND) rows += add[i];
            pages += need[i];
        }
        const int64_t rows_here = EXTEND ? wave_sums(rows) : 0, pages_here = wave_sums(pages);
        if (lane == 63) {
            wave_total[0][wave] = rows_here;
            wave_total[1][wave] = pages_here;
        }
        __syncthreads();
        int64_t r = rows_before + rows_here - rows, p = pages_before + pages_here - pages;
        for (int w = 0; w < waves; ++w) {
            if (EXTEND) {
                r += w < wave ? wave_total[0][w] : 0;
                rows_before += wave_total[0][w];
            }
            p += w < wave ? wave_total[1][w] : 0;
            pages_before += wave_total[1][w];
        }
        if (EXTEND) {   // sums grow with the sequence: those that do not fit are the last ones
            int64_t re = r, pe = p;
            int over = a.sequences;
#pragma unroll
            for (int i = kPagesEach - 1; i >= 0; --i) {
                re = r, pe = p;
#pragma unroll
                for (int k = 0; k <= i; ++k) re += add[k], pe += need[k];
                if (base + t * kPagesEach + i < a.sequences && (re > a.rows || pe > top)) over = base + t * kPagesEach + i;
            }
            if (over < a.sequences) atomicMin(&lds_stop, over);
            __syncthreads();
            if (stop == a.sequences) stop = lds_stop;
        }
#pragma unroll
        for (int i = 0; i < kPagesEach; ++i) {
            const int s = base + t * kPagesEach + i;
            if (s >= a.sequences) break;
            const bool in = !EXTEND || s < stop;
            if (EXTEND && s == stop) {   // all sums from here on are those of the sequences served
                wave_total[0][0] = r;
                wave_total[1][0] = p;
            }
            if (in) {
                if (EXTEND) a.offsets[s] = (int32_t)r;
                if (SPREAD) {
                    if (EXTEND) lds_rows[s] = (int32_t)r;
                    lds_page[s] = (int32_t)p;
                    lds_first[s] = from[i];
                } else {
                    a.page_off[s] = (int32_t)p;
                    a.first[s] = from[i];
                }
                if (add[i]) a.lengths[s] = EXTEND ? n[i] + add[i] : n[i];
                r += add[i];
                p += need[i];
            }
        }
        __syncthreads();
        if (EXTEND && stop < a.sequences && stop >= base && stop < base + chunk) {
            rows_before = wave_total[0][0];
            pages_before = wave_total[1][0];
            __syncthreads();
        }
        if (EXTEND && stop < a.sequences) {
            for (int s = std::max(base, stop) + t; s < std::min(base + chunk, a.sequences); s += blockDim.x) {
                a.offsets[s] = (int32_t)rows_before;
                if (SPREAD) {
                    lds_rows[s] = (int32_t)rows_before;
                    lds_page[s] = (int32_t)pages_before;
                    lds_first[s] = 0;
                } else {
                    a.page_off[s] = (int32_t)pages_before;
                    a.first[s] = 0;
                }
            }
        }
    }
    if (t == 0) {
        if (EXTEND) {
            a.offsets[a.sequences] = (int32_t)rows_before;
            *a.served = stop;
            *a.free_count = top - (int)pages_before;
        } else {
            *a.free_count = (int)std::min<int64_t>(top + pages_before, a.n_pages);
        }
        if (SPREAD) {
            if (EXTEND) lds_rows[a.sequences] = (int32_t)rows_before;
            lds_page[a.sequences] = (int32_t)pages_before;
        } else {
            a.page_off[a.sequences] = (int32_t)pages_before;
            *a.top = top;
        }
    }
    if (SPREAD) {
        __syncthreads();
        const PagesView v{lds_rows, lds_page, lds_first, a.sequences, top, (int)pages_before, (int)rows_before};
        pages_spread<EXTEND>(a, v, t, blockDim.x);
    }
}

template <bool EXTEND>
__global__ __launch_bounds__(256) void pages_spread_kernel(PagesArgs a) {
    const PagesView v{a.offsets, a.page_off, a.first, a.sequences, *a.top, a.page_off[a.sequences],
                      EXTEND ? a.offsets[a.sequences] : 0};
    pages_spread<EXTEND>(a, v, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

}  // namespace exq

// =================================================================== host

using namespace exq;

namespace {

struct Array {
    const char* name;
    const void* p;
    size_t bytes;
};

// Alignment of every array, and that no two share memory: of what a launch
// writes, other threads of it read the rest.
exq_status check_arrays(const Array* x, int n) {
    for (int i = 0; i < n; ++i) {
        if (!x[i].p && x[i].bytes) return fail(EXQ_ERR_INVALID_ARG, "%s is NULL", x[i].name);
        if (!aligned(x[i].p, 4)) return fail(EXQ_ERR_INVALID_ARG, "%s is misaligned", x[i].name);
        for (int j = 0; j < i; ++j)
            if (x[i].bytes && x[j].bytes && ranges_meet(x[i].p, x[i].bytes, x[j].p, x[j].bytes))
                return fail(EXQ_ERR_INVALID_ARG, "%s and %s overlap", x[j].name, x[i].name);
    }
    return EXQ_OK;
}

exq_status check_pages_call(const PagesArgs& a) {
    if (a.sequences < 1 || a.width < 1) return fail(EXQ_ERR_INVALID_ARG, "table of %d x %d", a.sequences, a.width);
    if (a.stride < 0 || a.stride > kMaxStride || (a.sequences > 1 && a.stride < a.width))
        return fail(EXQ_ERR_INVALID_ARG, "table_stride=%lld", (long long)a.stride);
    if (a.page_size < 1) return fail(EXQ_ERR_INVALID_ARG, "page_size=%d", a.page_size);
    if (a.n_pages < 1) return fail(EXQ_ERR_INVALID_ARG, "n_pages=%d", a.n_pages);
    if (a.rows < 0) return fail(EXQ_ERR_INVALID_ARG, "rows=%d", a.rows);
    if ((int64_t)a.sequences * a.width > 0x7FFFFFFF)
        return fail(EXQ_ERR_UNSUPPORTED, "a table of %d x %d: over 2^31 - 1 pages", a.sequences, a.width);
    return EXQ_OK;
}

// Rows and table entries up to which the workgroup that looks through the
// sequences does the rest of the call too.
constexpr int64_t kPagesAlone = 4096;

template <bool EXTEND> exq_status pages_call(PagesArgs a, void* workspace, void* stream, const char* what) {
    a.page_off = static_cast<int32_t*>(workspace);
    a.first = a.page_off + a.sequences + 1;
    a.top = a.first + a.sequences;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    // what there may be to do beside the look through the sequences: a page or two of each
    // and the rows of them, or all that is in the table
    const int64_t most = EXTEND ? std::max<int64_t>(a.rows, a.sequences) : (int64_t)a.sequences * a.width;
    const bool small = a.sequences <= 256 * kPagesEach && most <= 1024;
    const dim3 threads(small ? 256 : kPagesThreads);
    if (most <= kPagesAlone && a.sequences <= kPagesChunk) {
        hipLaunchKernelGGL((pages_scan_kernel<EXTEND, true>), dim3(1), threads, 0, s, a);
        return launched(what);
    }
    hipLaunchKernelGGL((pages_scan_kernel<EXTEND, false>), dim3(1), threads, 0, s, a);
    const exq_status st = launched(what);
    if (st != EXQ_OK) return st;
    hipLaunchKernelGGL((pages_spread_kernel<EXTEND>), dim3((unsigned)std::min<int64_t>((most + 255) / 256, 2048)), dim3(256), 0, s, a);
    return launched(what);
}

}  // namespace

extern "C" {

size_t exq_pages_workspace_bytes(int sequences) { return sequences < 1 ? 0 : 4 * (2 * (size_t)sequences + 2); }

exq_status exq_pages_extend(int32_t* table, int sequences, int table_width, int64_t table_stride, int page_size,
                            int32_t* lengths, const int32_t* counts, const int32_t* free_pages, int32_t* free_count,
                            int n_pages, int32_t* seqs, int32_t* positions, int rows, int32_t* offsets, int32_t* served,
                            void* workspace, size_t workspace_bytes, void* stream) {
    PagesArgs a{table, table_stride, sequences, table_width, page_size, lengths, counts, const_cast<int32_t*>(free_pages),
                free_count, n_pages, seqs, positions, offsets, served, rows, nullptr, nullptr, nullptr};
    exq_status st = check_pages_call(a);
    if (st != EXQ_OK) return st;
    const size_t n = 4 * (size_t)sequences, need = exq_pages_workspace_bytes(sequences);
    if (workspace_bytes < need) return fail(EXQ_ERR_INVALID_ARG, "workspace of %zu bytes: %zu are needed", workspace_bytes, need);
    const Array arrays[] = {{"table", table, table_extent(sequences, table_width, table_stride)}, {"lengths", lengths, n},
                            {"counts", counts, n}, {"free_pages", free_pages, 4 * (size_t)n_pages}, {"free_count", free_count, 4},
                            {"seqs", seqs, 4 * (size_t)rows}, {"positions", positions, 4 * (size_t)rows},
                            {"offsets", offsets, n + 4}, {"served", served, 4}, {"workspace", workspace, need}};
    if ((st = check_arrays(arrays, 10)) != EXQ_OK) return st;
    return pages_call<true>(a, workspace, stream, "pages extend launch");
}

exq_status exq_pages_trim(int32_t* table, int sequences, int table_width, int64_t table_stride, int page_size,
                          int32_t* lengths, const int32_t* keep, int32_t* free_pages, int32_t* free_count, int n_pages,
                          void* workspace, size_t workspace_bytes, void* stream) {
    PagesArgs a{table, table_stride, sequences, table_width, page_size, lengths, keep, free_pages,
                free_count, n_pages, nullptr, nullptr, nullptr, nullptr, 0, nullptr, nullptr, nullptr};
    exq_status st = check_pages_call(a);
    if (st != EXQ_OK) return st;
    const size_t n = 4 * (size_t)sequences, need = exq_pages_workspace_bytes(sequences);
    if (workspace_bytes < need) return fail(EXQ_ERR_INVALID_ARG, "workspace of %zu bytes: %zu are needed", workspace_bytes, need);
    const Array arrays[] = {{"table", table, table_extent(sequences, table_width, table_stride)}, {"lengths", lengths, n},
                            {"keep", keep, n}, {"free_pages", free_pages, 4 * (size_t)n_pages}, {"free_count", free_count, 4},
                            {"workspace", workspace, need}};
    if ((st = check_arrays(arrays, 6)) != EXQ_OK) return st;
    return pages_call<false>(a, workspace, stream, "pages trim launch");
}

}  // extern "C"
