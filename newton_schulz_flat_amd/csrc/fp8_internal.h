// Internal declarations of the casts into 8-bit blocks and of their products.
// Like clipping they keep no plan: all that a kernel has to know travels in its
// arguments.
#pragma once

#include "muon_internal.h"

namespace muon {

constexpr int kFp8Block = 128;  // elements of a block along a row
constexpr int64_t kFp8MaxSide = int64_t(1) << 24;
constexpr int64_t kFp8MaxOut = int64_t(1) << 36;

inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

hipError_t launch_fp8_cast(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride,
                           const muon_fp8_t* out, const muon_fp8_t* out_t, hipStream_t s);

// Workspace bytes of a product.
size_t fp8_workspace_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_fp8_matmul(const muon_fp8_t& a, const muon_fp8_t& b, void* out, int out_dtype,
                             int64_t out_row_stride, bool accumulate, void* workspace,
                             hipStream_t s);

}  // namespace muon
