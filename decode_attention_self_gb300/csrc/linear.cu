// Matrix product with an epilogue: which kernel takes a call, and the tensor maps that they share.
#include <stdlib.h>
#include <cudaTypedefs.h>

#include "dr_layer.h"

namespace dr {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *ptr = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

}  // namespace

bool encode_matrix(CUtensorMap *map, const void *ptr, bool f32, int64_t rows, int cols, int64_t stride, int box_rows,
                   int box_cols) {
    const auto enc = tensor_map_encoder();
    if (!enc) return false;
    const int e = f32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * e};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               box_cols * e == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// Prompts go to the pairs of CTAs.
bool takes_tiles(const LinearParams &p, int sms) {
    const int64_t tiles = linear_tiles_tiles(p, sms);
    if (getenv("LCL")) return !atoi(getenv("LCL"));
    return tiles * 2 >= sms / 2;
}

}  // namespace

int linear_tiles(const LinearParams &p, int sms) {
    return takes_tiles(p, sms) ? linear_tiles_tiles(p, sms) : linear_cluster_tiles(p, sms);
}

cudaError_t launch_linear(const LinearParams &p, cudaStream_t stream) {
    const int sms = current_device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    return takes_tiles(p, sms) ? launch_linear_tiles(p, sms, stream) : launch_linear_cluster(p, sms, stream);
}

}  // namespace dr
