// decay_common.cuh -- what the calls of linear attention with a decay a head share:
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
//   g_t = min(head_decay[h] + log_decay[t, h], 0).
#pragma once

#include "latent_common.cuh"

namespace kda {

// One of the two at least, of whole floats (read one at a time, so that rows of log_decay may start anywhere).
inline bool decays_ok(const float* head_decay, const float* log_decay) {
    return (head_decay || log_decay) && reinterpret_cast<uintptr_t>(head_decay) % 4 == 0 && reinterpret_cast<uintptr_t>(log_decay) % 4 == 0;
}

// Log decay of row t and head h (either source may be missing).  Above 0 counts as 0, and below
// -104 (whose exponential is 0 in fp32), -inf included, as -104, so that differences of sums stay
// numbers; NaN stays NaN.
__device__ __forceinline__ float log_decay_of(const float* head_decay, const float* log_decay, int64_t t, int H, int h) {
    float g = 0.f;
    if (head_decay) g += head_decay[h];
    if (log_decay) g += log_decay[t * H + h];
    g = g > 0.f ? 0.f : g;
    return g < -104.f ? -104.f : g;
}

// Four consecutive elements of a row of any of the three types (index i % 4 == 0).
__device__ __forceinline__ float4 load4_as(const void* p, int64_t i, int dt) {
    if (dt == KDA_F32) return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
    const float2 a = dt == KDA_BF16 ? Elem<KDA_BF16>::get2(w.x) : Elem<KDA_F16>::get2(w.x);
    const float2 b = dt == KDA_BF16 ? Elem<KDA_BF16>::get2(w.y) : Elem<KDA_F16>::get2(w.y);
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float load1_as(const void* p, int64_t i, int dt) {
    if (dt == KDA_F32) return static_cast<const float*>(p)[i];
    if (dt == KDA_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store1_as(void* p, int64_t i, float x, int dt) {
    if (dt == KDA_F32) static_cast<float*>(p)[i] = x;
    else if (dt == KDA_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
    else static_cast<__half*>(p)[i] = __float2half_rn(x);
}

}  // namespace kda
