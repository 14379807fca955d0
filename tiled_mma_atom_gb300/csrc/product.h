// product.h — what the entry points of the products share on the host: argument
// checks, and the products themselves as steps of other calls (api_grouped.cu).
#pragma once

#include <exception>

#include "grouped.h"
#include "host.h"

namespace tmg {

constexpr int64_t kMax31 = (int64_t{1} << 31) - 1;

// No C++ exception leaves a C entry point.
template <class F>
tmg_status guarded(F &&body)
{
    try {
        clear_error();
        return body();
    } catch (const std::exception &x) {
        return fail(TMG_ERR_CUDA, "host error: %s", x.what());
    } catch (...) {
        return fail(TMG_ERR_CUDA, "host error");
    }
}

inline tmg_status launched(cudaError_t e, const char *what) { return e == cudaSuccess ? TMG_OK : cuda_fail(e, what); }

// (a - 1) * b + ... of a strided operand must stay within int64.
inline bool extents_ok(int64_t rows, int64_t row_stride, int64_t cols, int64_t col_stride, int64_t outer = 1, int64_t outer_stride = 0)
{
    if (row_stride < 0 || col_stride < 0 || outer_stride < 0)
        return false;
    const __int128 off = static_cast<__int128>(rows > 0 ? rows - 1 : 0) * row_stride +
                         static_cast<__int128>(cols > 0 ? cols - 1 : 0) * col_stride +
                         static_cast<__int128>(outer > 0 ? outer - 1 : 0) * outer_stride;
    return off < (static_cast<__int128>(1) << 60);
}

// An output's rows must not overlap.
inline bool out_rows_ok(int64_t rows, int64_t cols, int64_t ld) { return rows <= 1 || ld >= cols; }

inline bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether TMA reads a (rows, cols) operand of `elem`-byte elements in place:
// 16-byte aligned base and rows, strides below 2^40 bytes, and rows that do not overlap.
inline bool rows_in_place(const void *p, int64_t rows, int64_t row, int64_t cols, int64_t col, int elem)
{
    return aligned(p) && cols > 0 && rows > 0 && (cols == 1 || col == 1) &&
           (rows == 1 || (row >= cols && row * elem % 16 == 0 && row * elem < (int64_t{1} << 40)));
}

// A stride for a dimension of extent 1, where the caller's says nothing.
inline int64_t stride_or(int64_t extent, int64_t stride, int64_t least) { return extent > 1 ? stride : least; }

inline int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Copy an operand of E blocks (rows, K) to workspace `which` at `offset`
// bytes of `total`.
tmg_status pack(const DeviceState &ds, Workspace which, Pack3Args a, int elem, size_t total, int64_t offset, cudaStream_t s,
                char **out);
// The grouped or the dense product and the grouped weight gradient (a.R > 0), with
// the stream's lock held and arguments that have been checked.
tmg_status run_product(const DeviceState &ds, const GroupedArgs &a, cudaStream_t s);
tmg_status run_wgrad(const DeviceState &ds, const WgradArgs &a, cudaStream_t s);

}  // namespace tmg
