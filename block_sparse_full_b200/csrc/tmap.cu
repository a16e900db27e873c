// Tensor maps of strided bf16 tensors (tmap.h): the driver's encoder, looked up once.
#include "tmap.h"

#include <cudaTypedefs.h>

#include <mutex>

namespace ssa {

int make_map(CUtensorMap* m, void* ptr, int rank, const unsigned long long* dims, const long long* strides,
             const unsigned* box) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    if (!fn) return fail(SSA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    cuuint64_t d[5], st[4];
    cuuint32_t bx[5], es[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) d[i] = dims[i], bx[i] = box[i];
    for (int i = 0; i + 1 < rank; ++i) st[i] = (cuuint64_t)strides[i] * 2;
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, ptr, d, st, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SSA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return SSA_OK;
}

int make_view_map(CUtensorMap* m, const View& v, int D, int T, int H, int B, int rows) {
    const unsigned long long dims[4] = {(unsigned long long)D, (unsigned long long)T, (unsigned long long)H,
                                        (unsigned long long)B};
    const long long strides[3] = {v.st, v.sh, v.sb};
    const unsigned box[4] = {64, (unsigned)rows, 1, 1};
    return make_map(m, v.data, 4, dims, strides, box);
}

}  // namespace ssa
