// Tensor maps of strided bf16 tensors, for the kernels that load by TMA.
#pragma once

#include <cuda.h>

#include "ssa_internal.h"

namespace ssa {

// 4-D bf16 tensor of dims[0] contiguous elements; strides of dims 1..3 and the
// box in elements; 128-byte swizzle, zeros outside the tensor.
int make_map4(CUtensorMap* m, void* ptr, const unsigned long long (&dims)[4], const long long (&strides)[3],
              const unsigned (&box)[4]);

// A view [B, H, T, D] as (d, t, h, b) with boxes of 64 elements x `rows` tokens.
int make_view_map(CUtensorMap* m, const View& v, int D, int T, int H, int B, int rows);

}  // namespace ssa
