// latent_prefill.cu -- kda_latent_prefill: expanded latent attention, in its plain blocked form
// on the CUDA cores.
//
// A block owns 32 query rows (8 a warp) and walks its keys 32 at a time through shared memory
// with the running maximum and sum of a softmax: o = sum_p e^{s_p - m} v_p, l = sum_p e^{s_p - m}
// in registers, rescaled by e^{m - m'} when the maximum moves.
#include "kda_host.h"
#include "latent_common.cuh"
#include "latent_host.h"

namespace kda {
namespace {

struct PrefillArgs {
    LatentRows q, k, v;
    const uint16_t* kr;
    int64_t kr_stride;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int32_t N, Tq, Tk, H;
    float scale;
    int32_t full;
    void* out;
    int64_t out_rs, out_hs;
    int32_t out_dt;
    float* lse;
    int32_t* dev_status;
};

constexpr int kRowsB = 32, kKeysB = 32, kWarps = 4, kRowsW = kRowsB / kWarps;

// The walk over keys of one block.  qrow(i, d): query channel; key(p, d), val(p, d): channels of
// key p (only for p with ok(p)); last(i): last key row i sees; store(i, o[], lse).
template <int DK, int DV, class Q, class KF, class VF, class OK, class LAST, class ST>
__device__ void attend(float* sm, int rows, int n_keys, float scale, Q qrow, KF key, VF val, OK ok, LAST last, ST store) {
    float* sq = sm;                      // [32][DK]
    float* sk = sq + kRowsB * DK;        // [32][DK + 1]
    float* sv = sk + kKeysB * (DK + 1);  // [32][DV]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float inf = __int_as_float(0x7f800000);
    for (int e = tid; e < kRowsB * DK; e += kWarps * 32) sq[e] = e / DK < rows ? qrow(e / DK, e % DK) * scale : 0.f;
    float m[kRowsW], l[kRowsW], o[kRowsW][DV / 32];
#pragma unroll
    for (int i = 0; i < kRowsW; ++i) {
        m[i] = -inf;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < DV / 32; ++j) o[i][j] = 0.f;
    }
    for (int p0 = 0; p0 < n_keys; p0 += kKeysB) {
        __syncthreads();
        for (int e = tid; e < kKeysB * DK; e += kWarps * 32) {
            const int p = p0 + e / DK;
            sk[(e / DK) * (DK + 1) + e % DK] = p < n_keys && ok(p) ? key(p, e % DK) : 0.f;
        }
        for (int e = tid; e < kKeysB * DV; e += kWarps * 32) {
            const int p = p0 + e / DV;
            sv[e] = p < n_keys && ok(p) ? val(p, e % DV) : 0.f;
        }
        __syncthreads();
        const int p = p0 + lane;
        const bool pok = p < n_keys && ok(p);
#pragma unroll
        for (int i = 0; i < kRowsW; ++i) {
            const int row = warp * kRowsW + i;
            float s = 0.f;
            for (int d = 0; d < DK; ++d) s = fmaf(sq[row * DK + d], sk[lane * (DK + 1) + d], s);
            if (!pok || p > last(row)) s = -inf;
            float mx = s;
#pragma unroll
            for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, w));
            const float mn = fmaxf(m[i], mx);
            if (mn == -inf) continue;
            const float f = expf(m[i] - mn), e = expf(s - mn);
            m[i] = mn;
            l[i] = l[i] * f + warp_sum(e);
#pragma unroll
            for (int j = 0; j < DV / 32; ++j) o[i][j] *= f;
            for (int q = 0; q < kKeysB; ++q) {
                const float pq = __shfl_sync(~0u, e, q);
#pragma unroll
                for (int j = 0; j < DV / 32; ++j) o[i][j] = fmaf(pq, sv[q * DV + lane + 32 * j], o[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRowsW; ++i) {
        const int row = warp * kRowsW + i;
        if (row >= rows) continue;
        const float il = l[i] > 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
        for (int j = 0; j < DV / 32; ++j) store(row, lane + 32 * j, o[i][j] * il);
        if (lane == 0) store(row, -1, l[i] > 0.f ? m[i] + logf(l[i]) : -inf);
    }
}

__device__ __forceinline__ void put(void* out, int64_t i, float x, int dt) {
    if (dt == KDA_F32) static_cast<float*>(out)[i] = x;
    else if (dt == KDA_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(x);
    else static_cast<__half*>(out)[i] = __float2half_rn(x);
}

template <int DT>
__global__ void __launch_bounds__(128) prefill_kernel(const __grid_constant__ PrefillArgs a) {
    extern __shared__ float sm[];
    using E = Elem<DT>;
    auto ld = [](const uint16_t* p) { return E::get(*reinterpret_cast<const typename E::T*>(p)); };
    int tile = blockIdx.x, q0 = 0, q1 = 0, k0 = 0, k1 = 0, n = 0;
    for (; n < a.N; ++n) {
        q0 = a.cu_q[n], q1 = a.cu_q[n + 1], k0 = a.cu_k[n], k1 = a.cu_k[n + 1];
        if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk) {
            if (threadIdx.x == 0) report(a.dev_status, KDA_DEV_BAD_SEQLEN);
            continue;
        }
        const int tiles = (q1 - q0 + kRowsB - 1) / kRowsB;
        if (tile < tiles) break;
        tile -= tiles;
    }
    if (n == a.N) return;
    const int h = blockIdx.y, row0 = tile * kRowsB, rows = min(kRowsB, q1 - q0 - row0);
    auto ok = [&](int) { return true; };
    auto key = [&](int p, int d) {
        return d < kNope ? ld(a.k.base + (k0 + p) * a.k.rs + h * a.k.hs + d) : ld(a.kr + (k0 + p) * a.kr_stride + d - kNope);
    };
    auto val = [&](int p, int d) { return ld(a.v.base + (k0 + p) * a.v.rs + h * a.v.hs + d); };
    auto q = [&](int i, int d) { return ld(a.q.base + (q0 + row0 + i) * a.q.rs + h * a.q.hs + d); };
    const int off = a.full ? 1 << 30 : (k1 - k0) - (q1 - q0) + row0;
    auto last = [&](int i) { return off + i; };
    auto store = [&](int i, int d, float x) {
        const int64_t row = q0 + row0 + i;
        if (d >= 0) put(a.out, row * a.out_rs + h * a.out_hs + d, x, a.out_dt);
        else if (a.lse) a.lse[row * a.H + h] = x;
    };
    const int n_keys = a.full ? k1 - k0 : max(0, min(k1 - k0, off + rows));
    attend<kHeadK, kHeadV>(sm, rows, n_keys, a.scale, q, key, val, ok, last, store);
}

constexpr int smem_of(int dk, int dv) { return (kRowsB * dk + kKeysB * (dk + 1) + kKeysB * dv) * 4; }

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_latent_prefill(const kda_rows_desc* q, const kda_rows_desc* k_nope,
                                         const void* k_rope, int64_t k_rope_stride,
                                         const kda_rows_desc* v, kda_dtype in_dtype,
                                         const int32_t* cu_q, const int32_t* cu_k, int32_t N,
                                         int32_t Tq, int32_t Tk, int32_t H, int32_t d_nope,
                                         int32_t d_rope, int32_t dv, float scale, uint32_t flags,
                                         const kda_rows_desc* out, kda_dtype out_dtype, float* lse,
                                         int32_t* dev_status, void* stream) {
    KDA_REQUIRE(N >= 0 && Tq >= 0 && Tk >= 0 && H > 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(d_nope == kNope && d_rope == kRope && dv == kHeadV, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((in_dtype == KDA_BF16 || in_dtype == KDA_F16) && any_dtype_ok(out_dtype), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((flags & ~KDA_LATENT_FULL) == 0 && H < 65536, KDA_ERR_UNSUPPORTED);
    if (N == 0 || Tq == 0) return KDA_OK;
    KDA_REQUIRE(rows_ok(q) && rows_ok(out), KDA_ERR_INVALID_ARG);
    if (Tk > 0) {
        KDA_REQUIRE(rows_ok(k_nope) && rows_ok(v), KDA_ERR_INVALID_ARG);
        KDA_REQUIRE(k_rope != nullptr && aligned16(k_rope), KDA_ERR_INVALID_ARG);
    }
    KDA_REQUIRE(k_nope != nullptr && v != nullptr, KDA_ERR_INVALID_ARG);
    const void* ptrs[] = {cu_q, cu_k};
    for (const void* p : ptrs) KDA_REQUIRE(p != nullptr && aligned16(p), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(k_rope_stride % 8 == 0 && k_rope_stride >= kRope, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(aligned16(lse) && aligned16(dev_status), KDA_ERR_INVALID_ARG);
    const PrefillArgs a{as_rows(q), as_rows(k_nope), as_rows(v), static_cast<const uint16_t*>(k_rope), k_rope_stride,
                        cu_q, cu_k, N, Tq, Tk, H, scale, (flags & KDA_LATENT_FULL) != 0, const_cast<void*>(out->base),
                        out->row_stride, out->head_stride, out_dtype, lse, dev_status};
    const dim3 grid((unsigned)(Tq / kRowsB + N), (unsigned)H);
    constexpr int smem = smem_of(kHeadK, kHeadV);
    auto* f = in_dtype == KDA_BF16 ? prefill_kernel<KDA_BF16> : prefill_kernel<KDA_F16>;
    cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    f<<<grid, 128, smem, as_stream(stream)>>>(a);
    return launch_status();
}
