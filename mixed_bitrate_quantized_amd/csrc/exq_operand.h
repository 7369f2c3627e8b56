// Host-side checks shared by the entry points on tensors: alignment, strides,
// extents, overlaps, and the error of a launch.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "exq_internal.h"

namespace exq {

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// An fp16 operand of (rows, heads, head_dim) with element strides.
struct Operand {
    const char* name;
    const void* p;
    int64_t row, head;
    int rows, heads, dim;
};

constexpr int64_t kMaxStride = (int64_t)1 << 30;   // elements: with 2^31 rows and heads extents stay inside 64 bits

inline exq_status check_operand(const Operand& x) {
    if (!x.p) return fail(EXQ_ERR_INVALID_ARG, "%s is NULL", x.name);
    if (!aligned(x.p, 16)) return fail(EXQ_ERR_INVALID_ARG, "%s must be 16-byte aligned", x.name);
    if (x.row < 0 || x.head < 0 || x.row % 8 || x.head % 8 || x.row > kMaxStride || x.head > kMaxStride)
        return fail(EXQ_ERR_INVALID_ARG, "%s: strides (%lld, %lld) must be multiples of 8 in 0..2^30", x.name,
                    (long long)x.row, (long long)x.head);
    return EXQ_OK;
}

inline size_t extent(const Operand& x) {   // bytes from its first element to past its last
    return 2 * ((size_t)(x.rows - 1) * (size_t)x.row + (size_t)(x.heads - 1) * (size_t)x.head + (size_t)x.dim);
}

inline bool ranges_meet(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

// Whether no element of x is written twice.
inline bool distinct(const Operand& x) {
    const int64_t rows = x.rows, heads = x.heads, dim = x.dim;
    const bool rows_outer = (heads == 1 || x.head >= dim) && (rows == 1 || x.row >= (heads - 1) * x.head + dim);
    const bool heads_outer = (rows == 1 || x.row >= dim) && (heads == 1 || x.head >= (rows - 1) * x.row + dim);
    return rows_outer || heads_outer;
}

// Whether two operands may share memory.  Slices of one buffer's rows (equal
// row strides, disjoint within the row) do not, although their extents meet.
inline bool operands_meet(const Operand& a, const Operand& b) {
    if (!ranges_meet(a.p, extent(a), b.p, extent(b))) return false;
    if (a.row != b.row || a.row == 0) return true;
    const int64_t stride = 2 * a.row, na = 2 * ((a.heads - 1) * a.head + a.dim), nb = 2 * ((b.heads - 1) * b.head + b.dim);
    const int64_t diff = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
    const int64_t at = ((diff % stride) + stride) % stride;   // where b's rows start within a's stride
    return !(na <= at && at + nb <= stride);
}

inline exq_status check_table(const int32_t* table, int rows, int width, int64_t stride) {
    if (!table || !aligned(table, 4)) return fail(EXQ_ERR_INVALID_ARG, "table is NULL or misaligned");
    if (rows < 1 || width < 1) return fail(EXQ_ERR_INVALID_ARG, "table of %d x %d", rows, width);
    if (stride < 0 || stride > kMaxStride || (rows > 1 && stride != 0 && stride < width))
        return fail(EXQ_ERR_INVALID_ARG, "table_stride=%lld", (long long)stride);
    return EXQ_OK;
}

// Bytes of a table from its first element to past its last.
inline size_t table_extent(int rows, int width, int64_t stride) {
    return 4 * ((size_t)(rows - 1) * (size_t)stride + (size_t)width);
}

constexpr int64_t kMaxLaunchThreads = 0xFFFFFFFFll;

inline exq_status launched(const char* what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? EXQ_OK : fail(EXQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

}  // namespace exq
