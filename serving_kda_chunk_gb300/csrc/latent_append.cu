// latent_append.cu -- kda_latent_append: latent vectors (normalised) and rope keys of new
// tokens into a paged cache.
//
// A warp per token: lane l holds 16 of the 512 latent channels (two 16-byte words) and, for
// l < 8, 8 of the 64 rope channels; the mean square is a warp sum in fp32 and every result is
// rounded once.  It moves 1152 bytes in and 1152 out a token and nothing else, so HBM sets its floor: 14.1 us
// for 41460 tokens.  It takes 21.8, since a warp's loads, sum and stores follow one another once and only the
// other blocks of an SM run under them.
#include "kda_host.h"
#include "latent_common.cuh"

namespace kda {
namespace {

struct AppendArgs {
    const uint16_t* kv;
    int64_t kv_stride;
    const uint16_t* weight;
    float eps;
    int32_t T;
    const int32_t* slot;
    uint16_t* cache;
    int64_t P;
    int32_t page_size;
    int64_t page_stride;
    int32_t* dev_status;
};

constexpr int kAppendWarps = 4;

template <int DT>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const __grid_constant__ AppendArgs a) {
    using E = Elem<DT>;
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    // the place, the row and the weights are asked for together: the row does not wait for the place
    const int32_t slot = a.slot[t];
    const uint4* src = reinterpret_cast<const uint4*>(a.kv + t * a.kv_stride);
    uint4 w[2] = {__ldcs(src + lane), __ldcs(src + 32 + lane)};
    uint4 r = make_uint4(0, 0, 0, 0);
    if (lane < kRope / 8) r = __ldcs(src + kLatent / 8 + lane);
    uint4 g[2] = {r, r};
    if (a.weight != nullptr) {
        const uint4* wt = reinterpret_cast<const uint4*>(a.weight);
        g[0] = __ldg(wt + lane);
        g[1] = __ldg(wt + 32 + lane);
    }
    if (slot < 0) return;
    const int32_t page = slot / a.page_size;
    if (page >= a.P) {
        if (lane == 0) report(a.dev_status, KDA_DEV_BAD_SLOT);
        return;
    }
    uint4* dst = reinterpret_cast<uint4*>(a.cache + (int64_t)page * a.page_stride +
                                          (int64_t)(slot - page * a.page_size) * kLatentRow);
    if (a.weight != nullptr) {
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(&w[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = E::get2(p[j]);
                sq = fmaf(x.x, x.x, fmaf(x.y, x.y, sq));
            }
        }
        const float f = rsqrtf(warp_sum(sq) * (1.f / kLatent) + a.eps);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t* p = reinterpret_cast<uint32_t*>(&w[i]);
            const uint32_t* q = reinterpret_cast<const uint32_t*>(&g[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = E::get2(p[j]), y = E::get2(q[j]);
                p[j] = E::put2(x.x * f * y.x, x.y * f * y.y);
            }
        }
    }
    dst[lane] = w[0];
    dst[32 + lane] = w[1];
    if (lane < kRope / 8) dst[kLatent / 8 + lane] = r;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_latent_append(const void* kv, int64_t kv_stride, const void* weight,
                                        float eps, kda_dtype dtype, int32_t T, int32_t d_latent,
                                        int32_t d_rope, const int32_t* slot, void* cache, int64_t P,
                                        int32_t page_size, int64_t page_stride, int32_t* dev_status,
                                        void* stream) {
    KDA_REQUIRE(T >= 0 && P >= 0 && page_size > 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(d_latent == kLatent && d_rope == kRope, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(dtype == KDA_BF16 || dtype == KDA_F16, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(page_size % 8 == 0, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(kv_stride % 8 == 0 && kv_stride >= kLatentRow, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(page_stride % 8 == 0 && page_stride >= (int64_t)page_size * kLatentRow, KDA_ERR_INVALID_ARG);
    if (T == 0) return KDA_OK;
    const void* ptrs[] = {kv, slot};
    for (const void* p : ptrs) KDA_REQUIRE(p != nullptr && aligned16(p), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE((P == 0 || cache != nullptr) && aligned16(cache), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(aligned16(weight) && aligned16(dev_status), KDA_ERR_INVALID_ARG);
    const AppendArgs a{static_cast<const uint16_t*>(kv), kv_stride, static_cast<const uint16_t*>(weight), eps, T,
                       slot, static_cast<uint16_t*>(cache), P, page_size, page_stride, dev_status};
    const unsigned grid = (unsigned)((T + kAppendWarps - 1ll) / kAppendWarps);
    if (dtype == KDA_BF16)
        append_kernel<KDA_BF16><<<grid, kAppendWarps * 32, 0, as_stream(stream)>>>(a);
    else
        append_kernel<KDA_F16><<<grid, kAppendWarps * 32, 0, as_stream(stream)>>>(a);
    return launch_status();
}
