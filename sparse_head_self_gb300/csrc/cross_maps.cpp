// Tensor maps of head tensors (see cross_tiles.cuh).
#include <cuda.h>

#include "cross_tiles.cuh"

namespace fibatt {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// From the driver through the runtime's entry-point query, so that the
// library needs no link against libcuda; null if unavailable.
EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

}  // namespace

bool make_tensor(TensorArg *t, const fibatt_heads &v, int B, int H, int N, int rows, int heads,
                 fibatt_dtype dtype, bool swizzle) {
    const EncodeTiledFn f = encode_tiled();
    if (!f) return false;
    const int64_t stride[3] = {v.stride_n, v.stride_h, v.stride_b};
    const int size[3] = {N, H, B};
    int rows_step = 1, *step[3] = {&rows_step, &t->head_step, &t->seq_step};
    const cuuint64_t size_of = dtype == FIBATT_F32 ? 4 : 2;
    cuuint64_t dims[4] = {64, 1, 1, 1}, strides[3] = {64 * size_of, 64 * size_of, 64 * size_of};
    for (int i = 0; i < 3; ++i) {
        const bool wide = size[i] > 1 && stride[i] > 0;
        *step[i] = wide ? 1 : 0;
        if (!wide) continue;
        dims[i + 1] = (cuuint64_t)size[i];
        strides[i] = (cuuint64_t)stride[i] * size_of;
    }
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, (cuuint32_t)heads, 1}, estr[4] = {1, 1, 1, 1};
    const auto encode = [&] {
        return f(&t->map, dtype == FIBATT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.ptr, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = encode();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        // the first call of a thread whose device the runtime has not made current yet
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
        r = encode();
    }
    return r == CUDA_SUCCESS;
}

}  // namespace fibatt
