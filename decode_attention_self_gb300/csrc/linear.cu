// Matrix product with an epilogue: which kernel takes a call, and the tensor maps that they share.
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

enum class Way { kRows, kCluster, kTiles };

// Which kernel takes a call; measured on both sides of each border, us.
// Rows or cluster: 16 tokens 8192 -> 8192 24.6 and 27.8, 4096 -> 1024 5.2 and 6.2; 32 tokens, where a CTA's tokens weigh more, 1024 ->
// 1536 3.6 and 4.4, 1024 -> 4096 4.6 and 5.6, 4096 -> 1024 7.0 and 6.3, 1536 -> 6144 10.0 and 7.8, 8192 -> 8192 44 and 28.  (The rule
// looks at the weights' size alone and takes 4096 -> 1024 to the rows too.)
// Cluster or tiles: the pairs that stay take what is more than one wave of tiles of 128 tokens by 64 weight rows and, with bf16
// outputs, of pairs' tiles of 256 by 128.  1024 tokens 4096 -> 1024 (128 of 128 by 64) 12.6 and 18, 256 tokens 1024 -> 4096 (128) 6.7 and
// 8.3; 512 tokens 1024 -> 4096 (64 of 256 by 128) 7.9 and 9.7, 2048 tokens 4096 -> 1024 (64) 14.9 and 19.3, 700 tokens 1024 -> 4096 (96)
// 13.6 and 10.9; fp32 outputs, to pairs' tiles: 1024 tokens 1024 -> 1536 (48) with a residual 10.9 and 9.3, without one 9.5 and 9.1, 2048
// tokens 1024 -> 1024 (64) 9.8 and 9.6, 8.0 and 9.1.  (The rule does not look at the residual: what has none loses up to a tenth by it.)
// So do fp32 outputs of a K too long for the other kernel's short sums, and 17 to 128 tokens of more weight rows than a wave of 64 each
// takes (9728 on 152 SMs): tiles of 256 tokens are mostly empty there, and 9792 rows, 77 tiles of 128 for 76 pairs, go as 39 tiles of 256
// (64 tokens 1024 -> 9728 6.7 on this side, -> 9792 10.4 on the other).
Way way_of(const LinearParams &p, int sms) {
    const int64_t rows = (int64_t)p.N * (p.gated ? 2 : 1);
    if (p.T <= 16 || (p.T <= 32 && rows * p.K <= 6 << 20)) return Way::kRows;
    return linear_cluster_takes(p, sms) ? Way::kCluster : Way::kTiles;
}

}  // namespace

int linear_tiles(const LinearParams &p, int sms) {
    switch (way_of(p, sms)) {
        case Way::kRows: return 0;
        case Way::kCluster: return linear_cluster_tiles(p, sms);
        default: return linear_tiles_tiles(p, sms);
    }
}

cudaError_t launch_linear(const LinearParams &p, cudaStream_t stream) {
    const int sms = current_device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    switch (way_of(p, sms)) {
        case Way::kRows: return launch_linear_rows(p, sms, stream);
        case Way::kCluster: return launch_linear_cluster(p, sms, stream);
        default: return launch_linear_tiles(p, sms, stream);
    }
}

}  // namespace dr
