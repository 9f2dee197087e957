// latent_host.h -- host-side helpers of the latent attention entry points.
#pragma once

#include <math.h>

#include "kda_host.h"

namespace kda {

// Rows of heads as the kernels take them (strides in elements).
struct LatentRows {
    const uint16_t* base;
    int64_t rs, hs;
};

inline bool rows_ok(const kda_rows_desc* d) {
    return d != nullptr && d->base != nullptr && aligned16(d->base) && d->row_stride % 8 == 0 && d->head_stride % 8 == 0;
}
inline LatentRows as_rows(const kda_rows_desc* d) {
    return {static_cast<const uint16_t*>(d->base), d->row_stride, d->head_stride};
}
inline bool any_dtype_ok(kda_dtype d) { return d == KDA_BF16 || d == KDA_F16 || d == KDA_F32; }

// |scale| log2 e, for exponentials to base 2 of |scale| s (a negative scale negates an operand of
// s).  A zero scale becomes the least factor that keeps a masked -inf at -inf and every s at 0.
inline float log2_scale(float scale) {
    const float c = fabsf(scale) * 1.4426950408889634f;
    return c > 1e-37f ? c : 1e-37f;
}

// The largest power of two that divides n, at most `most`.
inline int lowbit_box(int n, int most) {
    int b = 1;
    while (b < most && n % (2 * b) == 0) b *= 2;
    return b;
}

// Tensor map over 16-bit elements, 128-byte swizzle, element strides 1.
inline bool encode_16bit(CUtensorMap* map, kda_dtype dt, int rank, const void* base, const cuuint64_t* dims,
                         const cuuint64_t* strides, const cuuint32_t* box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    return enc(map, dt == KDA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
               const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kda
