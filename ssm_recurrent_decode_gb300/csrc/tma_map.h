// tma_map.h -- tensor maps of head rows for TMA copies (internal to libgdn_decode.so).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>

namespace gdn {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
            fn.store(f, std::memory_order_release);
        } else {
            cudaGetLastError();
        }
    }
    return f;
}

// bf16 rows [T, heads, dim] (strides in elements) in boxes of `rows` tokens x 64 channels of one head, 128-byte
// swizzle, zeros outside. False where TMA cannot copy them: base or strides not multiples of 16 bytes.
inline bool encode_head_rows(CUtensorMap *map, const void *base, int T, int heads, int dim, int64_t stride, int64_t head, int rows)
{
    const auto fn = tensor_map_encoder();
    if (heads == 1) head = (dim + 7) / 8 * 8;
    if (T == 1) stride = (dim + 7) / 8 * 8;
    if (!fn || T < 1 || reinterpret_cast<uintptr_t>(base) % 16 || stride % 8 || head % 8 || stride <= 0 || head <= 0 ||
        stride >= (int64_t)1 << 38 || head >= (int64_t)1 << 38)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    const cuuint32_t one[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gdn
