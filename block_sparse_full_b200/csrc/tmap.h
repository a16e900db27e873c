// Tensor maps of strided bf16 tensors, for the kernels that load by TMA.
#pragma once

#include <cuda.h>

#include "ssa_internal.h"

namespace ssa {

// bf16 tensor of up to five axes, dims[0] elements contiguous; strides of the axes
// from 1 on and the box in elements; 128-byte swizzle, zeros outside the tensor.
int make_map(CUtensorMap* m, void* ptr, int rank, const unsigned long long* dims, const long long* strides,
             const unsigned* box);

// A view [B, H, T, D] as (d, t, h, b) with boxes of 64 elements x `rows` tokens.
int make_view_map(CUtensorMap* m, const View& v, int D, int T, int H, int B, int rows);

}  // namespace ssa
