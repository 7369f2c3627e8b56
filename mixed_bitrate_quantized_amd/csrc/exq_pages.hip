// Pages of a key-value cache handed out to sequences and taken back on the GPU
// (exq_pages_extend, exq_pages_trim), with the sequence and position of every
// new row.  include/exq.h says what they compute.
//
// Both are a prefix sum over the sequences, of the pages that move and of the
// new rows, and then one look-up for every page and row: the sequence whose
// range holds it.  Nothing is ordered by atomics, so the same inputs give the
// same pages.
//
// Bytes are few (1024 sequences with 4096 new rows: 64 KB); what a call costs is
// its launch, three dependent looks at memory (free_count, lengths, free_pages)
// and a search of log2(sequences) steps in LDS for every four rows.  On the GPU,
// trimming 16 sequences takes 2.3 us and 1024 (one launch) 3.6, adding 5 tokens to
// each of 16 takes 3.4 and up to 8 to each of 1024 6.2.
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
    bool vectors;            // seqs and positions are 16-byte aligned
    bool alone;              // no second launch follows
    // [sequences + 1] pages before each sequence's, [sequences] its tokens before the
    // new ones (extend) or left (trim), and the free list's count before the call
    int32_t *page_off, *start, *top;
};

constexpr int kPagesThreads = 1024;
constexpr int kPagesEach = 4;                             // sequences of a thread in one pass, at most
constexpr int kPagesChunk = kPagesThreads * kPagesEach;   // sequences of one pass

__device__ __forceinline__ int pages_of(int64_t tokens, int page_size) {
    return tokens <= 0 ? 0 : (int)((uint32_t)(tokens - 1) / (uint32_t)page_size) + 1;
}

// What the spreading half of a call looks things up in: prefix sums in LDS if one
// pass held them all, else in memory.
struct PagesView {
    const int32_t *rows_off, *page_off, *start;
    int sequences, top, pages, rows;
};

// The last s of [0, n) with off[s] <= x (off[0] = 0, ascending, x below off[n]):
// the one whose range [off[s], off[s + 1]) holds x.
__device__ __forceinline__ int holder(const int32_t* off, int n, int x) {
    int lo = 0, hi = n;   // off[lo] <= x < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Pages first, first + step, .. of a call, and rows four by four.
template <bool EXTEND>
__device__ __forceinline__ void pages_spread(const PagesArgs& a, const PagesView& v, int64_t first, int64_t step) {
    const int64_t most = std::min<int64_t>((int64_t)a.width * a.page_size, 0x7FFFFFFF);
    for (int64_t j = first; j < v.pages; j += step) {
        const int s = holder(v.page_off, v.sequences, (int)j);
        const int column = pages_of(std::min<int64_t>(v.start[s], most), a.page_size) + ((int)j - v.page_off[s]);
        int32_t* entry = a.table + (int64_t)s * a.stride + column;
        if (EXTEND) {
            *entry = a.free_pages[v.top - 1 - (int)j];
        } else {
            const int64_t to = (int64_t)v.top + v.pages - 1 - j;
            if (to < a.n_pages) a.free_pages[to] = *entry;
            *entry = -1;
        }
    }
    if (!EXTEND) return;
    typedef int32_t i4 __attribute__((ext_vector_type(4)));
    for (int64_t r0 = 4 * first; r0 < a.rows; r0 += 4 * step) {
        i4 seqs = {-1, -1, -1, -1}, positions = {0, 0, 0, 0};
        if (r0 < v.rows) {
            int s = holder(v.rows_off, v.sequences, (int)r0);
            int next = v.rows_off[s + 1], shift = v.start[s] - v.rows_off[s];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = (int)r0 + e;
                if (r >= v.rows) break;
                if (r >= next) {   // the next sequence that has rows
                    do next = v.rows_off[++s + 1];
                    while (r >= next);
                    shift = v.start[s] - v.rows_off[s];
                }
                seqs[e] = s;
                positions[e] = shift + r;
            }
        }
        if (a.vectors && r0 + 4 <= a.rows) {
            *gptr_w<i4>(a.seqs + r0) = seqs;
            *gptr_w<i4>(a.positions + r0) = positions;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r0 + e < a.rows) {
                    a.seqs[r0 + e] = seqs[e];
                    a.positions[r0 + e] = positions[e];
                }
        }
    }
}

// Pages of a trim that the first launch moves though a second one follows, which then
// finds nothing: a trim and an extend of 1024 sequences in a table of 252 pages each
// take 12.5 us instead of 14.0 where 300 pages go back, 12.3 instead of 12.9 (in a
// graph) at 1024 pages, 13.5 both at 2048, 17.5 instead of 15.8 at 4096.
constexpr int kPagesHere = 2048;

// One workgroup looks through all sequences; with SPREAD, if LDS holds them, it also
// does the rest, or leaves it to the second launch.
template <bool EXTEND, bool SPREAD>
__global__ __launch_bounds__(kPagesThreads) void pages_scan_kernel(PagesArgs a) {
    __shared__ int32_t lds_rows[EXTEND && SPREAD ? kPagesChunk + 1 : 1];
    __shared__ int32_t lds_page[SPREAD ? kPagesChunk + 1 : 1], lds_start[SPREAD ? kPagesChunk : 1];
    __shared__ uint64_t wave_rows[16], wave_pages[16];
    __shared__ uint64_t cut_rows, cut_pages;
    __shared__ int lds_stop;
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t / 64), lane = t % 64;
    const int each = min((a.sequences + (int)blockDim.x - 1) / (int)blockDim.x, kPagesEach), chunk = blockDim.x * each;
    const int64_t most = std::min<int64_t>((int64_t)a.width * a.page_size, 0x7FFFFFFF);
    const int top = min(max(*a.free_count, 0), a.n_pages);
    uint64_t rows_before = 0, pages_before = 0;
    int stop = a.sequences;   // the first sequence that does not fit
    if (t < 16) wave_rows[t] = wave_pages[t] = 0;
    if (t == 0) lds_stop = a.sequences;
    __syncthreads();
#pragma unroll 1
    for (int base = 0; base < a.sequences; base += chunk) {
        int n[kPagesEach], add[kPagesEach], need[kPagesEach];
        uint64_t rows = 0, pages = 0;
#pragma unroll
        for (int i = 0; i < kPagesEach; ++i) {
            const int s = base + t * each + i;
            const bool in = i < each && s < a.sequences && stop == a.sequences;
            n[i] = in ? a.lengths[s] : -1;
            const int c = in ? a.change[s] : 0;
            add[i] = need[i] = 0;
            if (EXTEND) {
                add[i] = n[i] < 0 ? 0 : max(c, 0);
                // what does not fit the table counts as 2^32 - 1 pages, more than a list has
                const int64_t end = (int64_t)n[i] + add[i];
                need[i] = add[i] == 0 ? 0 : end > most ? -1 : pages_of(end, a.page_size) - pages_of(n[i], a.page_size);
                rows += (uint32_t)add[i];
            } else if (c >= 0 && c < n[i]) {
                add[i] = 1;   // the length changes
                const int64_t held = std::min<int64_t>(n[i], most);
                need[i] = pages_of(held, a.page_size) - pages_of(std::min<int64_t>(c, held), a.page_size);
                n[i] = c;
            }
            pages += (uint32_t)need[i];
        }
        const uint64_t rows_to = EXTEND ? prefix64(rows) : 0, pages_to = prefix64(pages);
        if (lane == 63) {
            wave_rows[wave] = rows_to;
            wave_pages[wave] = pages_to;
        }
        __syncthreads();
        const uint64_t wr = EXTEND ? prefix16(wave_rows[lane & 15]) : 0, wp = prefix16(wave_pages[lane & 15]);
        uint64_t r = rows_before + rows_to - rows + (wave ? lane_value(wr, wave - 1) : 0);
        uint64_t p = pages_before + pages_to - pages + (wave ? lane_value(wp, wave - 1) : 0);
        rows_before += lane_value(wr, 15);
        pages_before += lane_value(wp, 15);
        if (EXTEND && stop == a.sequences && (rows_before > (uint64_t)a.rows || pages_before > (uint64_t)top)) {
            // the first that does not fit: sums grow along the sequences
            uint64_t re = r, pe = p;
#pragma unroll
            for (int i = 0; i < kPagesEach; ++i) {
                re += (uint32_t)add[i];
                pe += (uint32_t)need[i];
                if (i < each && (re > (uint64_t)a.rows || pe > (uint64_t)top)) {
                    atomicMin(&lds_stop, base + t * each + i);
                    break;
                }
            }
            __syncthreads();
            stop = lds_stop;
            re = r, pe = p;
#pragma unroll
            for (int i = 0; i < kPagesEach; ++i) {
                if (i < each && base + t * each + i == stop) {   // the sums of the sequences served
                    cut_rows = re;
                    cut_pages = pe;
                }
                re += (uint32_t)add[i];
                pe += (uint32_t)need[i];
            }
            __syncthreads();
            rows_before = cut_rows;
            pages_before = cut_pages;
        }
#pragma unroll
        for (int i = 0; i < kPagesEach; ++i) {
            const int s = base + t * each + i;
            if (i >= each || s >= a.sequences) break;
            const bool in = !EXTEND || s < stop;
            const int32_t rows_at = (int32_t)(in ? r : rows_before), pages_at = (int32_t)(in ? p : pages_before);
            if (EXTEND) a.offsets[s] = rows_at;
            if (SPREAD) {
                if (EXTEND) lds_rows[s] = rows_at;
                lds_page[s] = pages_at;
                lds_start[s] = n[i];
            } else {
                a.page_off[s] = pages_at;
                a.start[s] = n[i];
            }
            if (in && add[i]) a.lengths[s] = EXTEND ? n[i] + add[i] : n[i];
            r += (uint32_t)add[i];
            p += (uint32_t)need[i];
        }
        __syncthreads();   // the waves' sums are read
    }
    if (t == 0) {
        if (EXTEND) {
            a.offsets[a.sequences] = (int32_t)rows_before;
            *a.served = stop;
            *a.free_count = top - (int)pages_before;
        } else {
            *a.free_count = (int)std::min<uint64_t>(top + pages_before, a.n_pages);
        }
        if (SPREAD) {
            if (EXTEND) lds_rows[a.sequences] = (int32_t)rows_before;
            lds_page[a.sequences] = (int32_t)pages_before;
        }
    }
    const bool here = SPREAD && (a.alone || (!EXTEND && pages_before <= kPagesHere));
    if (t == 0 && !a.alone) {
        a.page_off[a.sequences] = here ? 0 : (int32_t)pages_before;   // 0: nothing is left
        *a.top = top;
    }
    if (SPREAD) {
        __syncthreads();
        const PagesView v{lds_rows, lds_page, lds_start, a.sequences, top, (int)pages_before, (int)rows_before};
        if (here) {
            pages_spread<EXTEND>(a, v, t, blockDim.x);
        } else {
            for (int i = t; i < a.sequences; i += blockDim.x) {
                a.page_off[i] = lds_page[i];
                a.start[i] = lds_start[i];
            }
        }
    }
}

constexpr int kSpreadThreads = 256;

// The other half for calls of many pages or rows.  Prefix sums that fit go to LDS
// first: a search in memory is a chain of loads.
template <bool EXTEND>
__global__ __launch_bounds__(kSpreadThreads) void pages_spread_kernel(PagesArgs a) {
    __shared__ int32_t lds_rows[EXTEND ? kPagesChunk + 1 : 1], lds_page[kPagesChunk + 1], lds_start[kPagesChunk];
    PagesView v{a.offsets, a.page_off, a.start, a.sequences, *a.top, a.page_off[a.sequences], EXTEND ? a.offsets[a.sequences] : 0};
    const int64_t first = (int64_t)blockIdx.x * kSpreadThreads + threadIdx.x, step = (int64_t)gridDim.x * kSpreadThreads;
    // (nothing to do for this workgroup)
    if ((int64_t)blockIdx.x * kSpreadThreads >= std::max<int64_t>(v.pages, EXTEND ? ((int64_t)a.rows + 3) / 4 : 0)) return;
    if (a.sequences <= kPagesChunk) {
#pragma unroll 4   // (loads of four at once)
        for (int i = threadIdx.x; i < a.sequences; i += kSpreadThreads) {
            if (EXTEND) lds_rows[i] = a.offsets[i];
            lds_page[i] = a.page_off[i];
            lds_start[i] = a.start[i];
        }
        if (threadIdx.x == 0) {
            if (EXTEND) lds_rows[a.sequences] = v.rows;
            lds_page[a.sequences] = v.pages;
        }
        __syncthreads();
        const PagesView w{lds_rows, lds_page, lds_start, v.sequences, v.top, v.pages, v.rows};
        pages_spread<EXTEND>(a, w, first, step);
        return;
    }
    pages_spread<EXTEND>(a, v, first, step);
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

// Rows, or table entries, up to which the workgroup that looks through the
// sequences does the rest of the call too.  A second launch costs 2.5 to 3 us
// whatever it finds: adding 4 tokens to each of 1024 sequences and trimming none
// takes 10.8 us with one launch each and 17.5 with two, of 4096 sequences 24.8 and
// 38.5.  Against that stand calls that move every page a table has, 2 ns a page in
// one workgroup: a full table of 1024 x 8 is emptied in 14 us by one launch and 12
// by two, of 1024 x 16 in 22 and 12, of 1024 x 252 in 500 and 13.
constexpr int64_t kPagesAlone = 16384;

template <bool EXTEND> exq_status pages_call(PagesArgs a, void* workspace, void* stream, const char* what) {
    a.page_off = static_cast<int32_t*>(workspace);
    a.start = a.page_off + a.sequences + 1;
    a.top = a.start + a.sequences;
    a.vectors = aligned(a.seqs, 16) && aligned(a.positions, 16);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    // what there may be to do beside the look through the sequences: the rows and a page or
    // two of each sequence, or all that is in the table
    const int64_t most = EXTEND ? std::max<int64_t>(a.rows, a.sequences) : (int64_t)a.sequences * a.width;
    const bool fits = a.sequences <= kPagesChunk;
    a.alone = most <= kPagesAlone && fits;
    const dim3 threads(a.sequences <= 256 && ((EXTEND && !a.alone) || most <= 1024) ? 256 : kPagesThreads);
    if (fits) hipLaunchKernelGGL((pages_scan_kernel<EXTEND, true>), dim3(1), threads, 0, s, a);
    else hipLaunchKernelGGL((pages_scan_kernel<EXTEND, false>), dim3(1), threads, 0, s, a);
    const exq_status st = launched(what);
    if (st != EXQ_OK || a.alone) return st;
    const int64_t work = EXTEND ? std::max<int64_t>((a.rows + 3) / 4, a.sequences) : most;
    hipLaunchKernelGGL((pages_spread_kernel<EXTEND>), dim3((unsigned)std::min<int64_t>((work + kSpreadThreads - 1) / kSpreadThreads, 512)),
                       dim3(kSpreadThreads), 0, s, a);
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
                free_count, n_pages, seqs, positions, offsets, served, rows, false, false, nullptr, nullptr, nullptr};
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
                free_count, n_pages, nullptr, nullptr, nullptr, nullptr, 0, false, false, nullptr, nullptr, nullptr};
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
