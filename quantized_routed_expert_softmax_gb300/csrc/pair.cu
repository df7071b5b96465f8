// pair.cu -- the tensor-map encoder of the CTA-pair products, looked up in the driver at run time.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "pair.cuh"

namespace moe {

cudaError_t tensor_map(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, int rank, const void* base, const int64_t* dims,
                       const int64_t* strides, const int64_t* box) {
    static std::once_flag once;
    static cudaError_t status = cudaSuccess;
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    std::call_once(once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q{};
        status = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (status == cudaSuccess && (q != cudaDriverEntryPointSuccess || fn == nullptr)) status = cudaErrorNotSupported;
        if (status == cudaSuccess) encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    if (status != cudaSuccess) return status;
    cuuint64_t d[5], st[4];
    cuuint32_t b[5];
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = static_cast<cuuint64_t>(dims[i]);
        b[i] = static_cast<cuuint32_t>(box[i]);
        if (i + 1 < rank) st[i] = static_cast<cuuint64_t>(strides[i]);
    }
    const CUresult r = encode(m, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace moe
