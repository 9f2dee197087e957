// latent_common.cuh -- element types and shapes shared by the latent attention
// and log-probability kernels.
#pragma once

#include "kda_common.cuh"

namespace kda {

constexpr int kLatent = 512;                  // latent vector of a token
constexpr int kRope = 64;                     // rope key of a token
constexpr int kLatentRow = kLatent + kRope;   // one cache row
constexpr int kNope = 128;                    // a head's expanded key, without the rope part
constexpr int kHeadK = kNope + kRope;
constexpr int kHeadV = 128;

// Element types of these calls: bf16, fp16 and fp32, widened exactly on load and rounded once
// (to nearest even) on store.
template <int DT>
struct Elem;
template <>
struct Elem<KDA_BF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float get(T x) { return __bfloat162float(x); }
    static __device__ __forceinline__ float2 get2(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t put2(float a, float b) { return pack_bf16x2(a, b); }
};
template <>
struct Elem<KDA_F16> {
    using T = __half;
    static __device__ __forceinline__ float get(T x) { return __half2float(x); }
    static __device__ __forceinline__ float2 get2(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t put2(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct Elem<KDA_F32> {
    using T = float;
    static __device__ __forceinline__ float get(T x) { return x; }
};

__host__ __device__ constexpr int dtype_bytes(int dt) { return dt == KDA_F32 ? 4 : 2; }

// 2^x (relative error about 2^-22; -inf gives 0, results below the normal range 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A running sum of weights, a tile's at a time, with what its roundings left out (the exact error of an
// addition): a plain fp32 sum over 10^5 keys behind one far larger weight drifts by 2^-14, alike in each step.
struct WeightSum {
    float s = 0.f, e = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float t = s + x, b = t - s;
        e += (s - (t - b)) + (x - b);
        s = t;
    }
    __device__ __forceinline__ void scale(float f) {
        s *= f;
        e *= f;
    }
    __device__ __forceinline__ float total() const { return s + e; }
};

// Softmax weights are 2^(c s - b), b = log2_base(m): the row's running maximum m in log2 units, m being up to
// 8 behind the largest score.  For fp16 products b is 7 lower, so that weights end at 2^15 (65504 is the
// largest fp16) and begin at 2^-32 of the row's largest: without it they began at 2^-25, and 10^5 keys some
// 25 below one other lost all their weight in the output but not in the sum.  bf16 has fp32's exponents.
// The sum of the weights has the same base, so lse = (b + log2 sum) ln 2.
template <int DT>
__device__ __forceinline__ float log2_base(float m, float c) {
    return DT == KDA_F16 ? fmaf(m, c, -7.f) : m * c;
}

// Four consecutive fp32 results (index i % 4 == 0) rounded into an output of type dt.
__device__ __forceinline__ void store4_as(void* p, int64_t i, float4 x, int dt) {
    if (dt == KDA_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = x;
    else if (dt == KDA_BF16)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) =
            make_uint2(Elem<KDA_BF16>::put2(x.x, x.y), Elem<KDA_BF16>::put2(x.z, x.w));
    else
        *reinterpret_cast<uint2*>(static_cast<__half*>(p) + i) =
            make_uint2(Elem<KDA_F16>::put2(x.x, x.y), Elem<KDA_F16>::put2(x.z, x.w));
}

}  // namespace kda
