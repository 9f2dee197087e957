// logprobs.cu -- kda_token_logprobs: log probability of given tokens, entropy and top
// alternatives of logits rows.
//
// A block per row.  Every thread keeps a running maximum m and, relative to it, z = sum e^{x-m}
// and w = sum e^{x-m} (x-m) over its elements; the block joins them, so
//   logprob = (x_token - m) - log z,  entropy = log z - w / z.
// The top ids are taken one after another: the largest (value, -id) below the last one taken.
#include "kda_host.h"
#include "latent_common.cuh"

namespace kda {
namespace {

struct LogprobArgs {
    const void* logits;
    int64_t row_stride;
    int32_t V;
    const int32_t* tokens;
    float* logprob;
    float* entropy;
    int32_t top;
    int32_t* top_ids;
    float* top_logprobs;
    int32_t* dev_status;
};

// (value, id) as one unsigned key: larger value first, then smaller id; -0 equals +0 and NaN
// lies below -inf.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t id) {
    const uint32_t b = __float_as_uint(x + 0.f);
    uint32_t o = (b & 0x80000000u) ? ~b : b | 0x80000000u;
    if (x != x) o = 0;
    return ((uint64_t)o << 32) | (uint32_t)~id;
}

constexpr int kLpThreads = 256;

template <int DT>
__global__ void __launch_bounds__(kLpThreads) logprob_kernel(const __grid_constant__ LogprobArgs a) {
    using E = Elem<DT>;
    __shared__ float sm[kLpThreads], sz[kLpThreads], sw[kLpThreads];
    __shared__ uint64_t sk[kLpThreads];
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    const typename E::T* row = static_cast<const typename E::T*>(a.logits) + r * a.row_stride;
    const float inf = __int_as_float(0x7f800000);
    float m = -inf, z = 0.f, w = 0.f;
    for (int i = tid; i < a.V; i += kLpThreads) {
        const float x = E::get(row[i]);
        if (x > m) {
            const float d = m - x, f = expf(d);
            w = z > 0.f ? f * (w + z * d) : 0.f;
            z *= f;
            m = x;
        }
        if (x != -inf) {
            const float d = x - m, e = expf(d);
            z += e;
            w += e > 0.f ? e * d : e;
        }
    }
    sm[tid] = m; sz[tid] = z; sw[tid] = w;
    __syncthreads();
    for (int s = kLpThreads / 2; s; s >>= 1) {
        if (tid < s) {
            const float m1 = sm[tid], m2 = sm[tid + s], mm = fmaxf(m1, m2);
            const float d1 = m1 - mm, d2 = m2 - mm;
            const float f1 = sz[tid] == 0.f ? 0.f : expf(d1), f2 = sz[tid + s] == 0.f ? 0.f : expf(d2);
            const float w1 = f1 == 0.f ? 0.f : f1 * (sw[tid] + sz[tid] * d1);
            const float w2 = f2 == 0.f ? 0.f : f2 * (sw[tid + s] + sz[tid + s] * d2);
            sw[tid] = w1 + w2;
            sz[tid] = f1 * sz[tid] + f2 * sz[tid + s];
            sm[tid] = mm;
        }
        __syncthreads();
    }
    m = sm[0]; z = sz[0]; w = sw[0];
    const float nan = __int_as_float(0x7fffffff);
    const bool none = !(z > 0.f) || m == inf;
    const float logz = none ? nan : logf(z);
    if (tid == 0) {
        const int tok = a.tokens[r];
        float lp = 0.f;
        if (tok >= a.V) report(a.dev_status, KDA_DEV_BAD_SLOT);
        else if (tok >= 0) lp = E::get(row[tok]) - m - logz;
        a.logprob[r] = lp;
        if (a.entropy) a.entropy[r] = logz - w / z;
    }
    uint64_t last = ~0ull;
    for (int j = 0; j < a.top; ++j) {
        uint64_t best = 0;
        for (int i = tid; i < a.V; i += kLpThreads) {
            const uint64_t k = order_key(E::get(row[i]), (uint32_t)i);
            if (k < last && k > best) best = k;
        }
        __syncthreads();
        sk[tid] = best;
        __syncthreads();
        for (int s = kLpThreads / 2; s; s >>= 1) {
            if (tid < s && sk[tid + s] > sk[tid]) sk[tid] = sk[tid + s];
            __syncthreads();
        }
        last = sk[0];
        if (tid == 0) {
            const int id = (int)~(uint32_t)last;
            a.top_ids[r * a.top + j] = id;
            a.top_logprobs[r * a.top + j] = E::get(row[id]) - m - logz;
        }
    }
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_token_logprobs(const void* logits, int64_t row_stride, kda_dtype dtype,
                                         int32_t R, int32_t V, const int32_t* tokens, float* logprob,
                                         float* entropy, int32_t top, int32_t* top_ids,
                                         float* top_logprobs, int32_t* dev_status, void* stream) {
    KDA_REQUIRE(R >= 0 && V > 0 && top >= 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(dtype == KDA_BF16 || dtype == KDA_F32 || dtype == KDA_F16, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(top <= 32 && top <= V, KDA_ERR_UNSUPPORTED);
    if (R == 0) return KDA_OK;
    KDA_REQUIRE(logits != nullptr && reinterpret_cast<uintptr_t>(logits) % dtype_bytes(dtype) == 0,
                KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(row_stride >= V || (R == 1 && row_stride >= 0), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(tokens != nullptr && logprob != nullptr, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(top == 0 || (top_ids != nullptr && top_logprobs != nullptr), KDA_ERR_INVALID_ARG);
    const void* ptrs[] = {tokens, logprob, entropy, top_ids, top_logprobs, dev_status};
    for (const void* p : ptrs) KDA_REQUIRE(aligned16(p), KDA_ERR_INVALID_ARG);
    const LogprobArgs a{logits, row_stride, V, tokens, logprob, entropy, top, top_ids, top_logprobs, dev_status};
    cudaStream_t s = as_stream(stream);
    if (dtype == KDA_BF16) logprob_kernel<KDA_BF16><<<(unsigned)R, kLpThreads, 0, s>>>(a);
    else if (dtype == KDA_F16) logprob_kernel<KDA_F16><<<(unsigned)R, kLpThreads, 0, s>>>(a);
    else logprob_kernel<KDA_F32><<<(unsigned)R, kLpThreads, 0, s>>>(a);
    return launch_status();
}
