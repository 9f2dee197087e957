// decay_prefill.cu -- kda_decay_prefill: linear attention with a decay a head over packed sequences.
//
// Token by token: a block holds 32 value channels of one (sequence, head) state in registers and walks the
// sequence, 16 tokens staged at a time.  The plainest right form; bound by its serial chain.
#include "decay_common.cuh"
#include "kda_host.h"
#include "latent_host.h"

#include <initializer_list>

namespace kda {
namespace {

constexpr int kDecayChunk = 128;

struct DecayPrefillArgs {
    LatentRows q, k, v, out;
    const float *head_decay, *log_decay;
    const int32_t *cu, *init_slot, *final_slot, *track_idx;
    void *pool, *track;
    int32_t* dev_status;
    int64_t P;
    int32_t N, T, H, group, M, in_dt, out_dt, st;
    float scale;
};

__global__ void __launch_bounds__(128) decay_serial_kernel(const DecayPrefillArgs a) {
    constexpr int TT = 16, RW = 8;
    __shared__ __align__(16) float sq[TT][kD], sk[TT][kD], sv[TT][32];
    __shared__ float dec[TT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.x & 3, unit = blockIdx.x >> 2;
    const int n = unit / a.H, h = unit - n * a.H, hk = h / a.group;
    const bool lead = threadIdx.x == 0 && part == 0 && h == 0;
    const int64_t first = a.cu[n], last = a.cu[n + 1];
    if (first < 0 || last < first || last > a.T) {
        if (lead) report(a.dev_status, KDA_DEV_BAD_SEQLEN);
        return;
    }
    const int64_t src = a.init_slot ? a.init_slot[n] : -1, dst = a.final_slot ? a.final_slot[n] : -1;
    if (src >= a.P || dst >= a.P) {
        if (lead) report(a.dev_status, KDA_DEV_BAD_SLOT);
        return;
    }
    const int row0 = part * 32 + warp * RW;
    const size_t at = (size_t)row0 * kD + 4 * lane;
    float4 s[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (src >= 0) s[i] = state_load4(a.pool, state_elem(src, a.H, h) + at + (size_t)i * kD, a.st);
    }
    const int64_t chunks = (last - first + kDecayChunk - 1) / kDecayChunk;
    for (int m = 0; lead && m < a.M; ++m) {
        const int c = a.track_idx[(int64_t)n * a.M + m];
        if (c < -1 || c >= chunks) report(a.dev_status, KDA_DEV_BAD_TRACK);
    }
    for (int64_t t0 = first; t0 < last; t0 += TT) {
        if ((t0 - first) % kDecayChunk == 0)
            for (int m = 0; m < a.M; ++m)
                if (a.track_idx[(int64_t)n * a.M + m] == (t0 - first) / kDecayChunk)
#pragma unroll
                    for (int i = 0; i < RW; ++i)
                        state_store4(a.track, state_elem((int64_t)n * a.M + m, a.H, h) + at + (size_t)i * kD, s[i], a.st);
        const int nt = (int)min((int64_t)TT, last - t0);
        __syncthreads();
        for (int t = warp; t < nt; t += 4) {
            auto row = [&](const LatentRows& d, int head) {
                return reinterpret_cast<const uint8_t*>(d.base) + ((t0 + t) * d.rs + head * d.hs) * 2;
            };
            const float4 q = load4_as(row(a.q, hk), 4 * lane, a.in_dt);
            *reinterpret_cast<float4*>(&sq[t][4 * lane]) = make_float4(q.x * a.scale, q.y * a.scale, q.z * a.scale, q.w * a.scale);
            *reinterpret_cast<float4*>(&sk[t][4 * lane]) = load4_as(row(a.k, hk), 4 * lane, a.in_dt);
            sv[t][lane] = load1_as(row(a.v, h), part * 32 + lane, a.in_dt);
        }
        if (threadIdx.x < nt) dec[threadIdx.x] = expf(log_decay_of(a.head_decay, a.log_decay, t0 + threadIdx.x, a.H, h));
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            const float4 k = *reinterpret_cast<const float4*>(&sk[t][4 * lane]);
            const float4 q = *reinterpret_cast<const float4*>(&sq[t][4 * lane]);
            float o = 0.f;
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                s[i] = f4_fma(sv[t][warp * RW + i], k, f4_mul(s[i], make_float4(dec[t], dec[t], dec[t], dec[t])));
                const float x = warp_sum(f4_dot(s[i], q));
                if (lane == i) o = x;
            }
            if (lane < RW) {
                void* p = const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(a.out.base) +
                                               ((t0 + t) * a.out.rs + h * a.out.hs) * dtype_bytes(a.out_dt));
                store1_as(p, row0 + lane, o, a.out_dt);
            }
        }
    }
    if (dst >= 0)
#pragma unroll
        for (int i = 0; i < RW; ++i) state_store4(a.pool, state_elem(dst, a.H, h) + at + (size_t)i * kD, s[i], a.st);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_decay_prefill_workspace_size(int32_t T_tot, int32_t N, int32_t H) {
    (void)T_tot, (void)N, (void)H;
    return 16;
}

extern "C" kda_status kda_decay_prefill(const kda_rows_desc* q, const kda_rows_desc* k, const kda_rows_desc* v,
                                        kda_dtype in_dtype, const float* head_decay, const float* log_decay,
                                        const int32_t* cu_seqlens, int32_t N, int32_t T_tot, int32_t H, int32_t Hk,
                                        int32_t dk, int32_t dv, float scale, uint32_t flags, void* state_pool, int64_t P,
                                        const int32_t* init_slot, const int32_t* final_slot,
                                        const int32_t* track_chunk_idx, int32_t M, void* track_state,
                                        const kda_rows_desc* out, kda_dtype out_dtype, void* workspace, size_t ws_bytes,
                                        int32_t* dev_status, void* stream) {
    KDA_REQUIRE(N >= 0 && T_tot >= 0 && H > 0 && Hk > 0 && P >= 0 && M >= 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(H % Hk == 0 && isfinite(scale), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(dk == kD && dv == kD, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((in_dtype == KDA_BF16 || in_dtype == KDA_F16) && any_dtype_ok(out_dtype), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((flags & ~(KDA_STATE_BF16 | KDA_STATE_F16)) == 0 && state_flags_ok(flags), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(T_tot < (1 << 30) && (int64_t)N * H < (1 << 27), KDA_ERR_UNSUPPORTED);
    if (N == 0) return KDA_OK;
    // without rows there is nothing to place, and states are passed on
    KDA_REQUIRE(T_tot == 0 || (rows_ok(q) && rows_ok(k) && rows_ok(v) && rows_ok(out)), KDA_ERR_INVALID_ARG);
    for (const kda_rows_desc* d : {q, k, v})
        KDA_REQUIRE(T_tot == 0 || ((d->row_stride > 0 || T_tot == 1) && d->head_stride >= 0), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(cu_seqlens && (head_decay || log_decay), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(state_pool || (!init_slot && !final_slot), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(M == 0 || (track_chunk_idx && track_state), KDA_ERR_INVALID_ARG);
    const void* ptrs[] = {cu_seqlens, head_decay, log_decay, state_pool, init_slot, final_slot, track_chunk_idx, track_state, workspace};
    for (const void* p : ptrs) KDA_REQUIRE(aligned16(p), KDA_ERR_INVALID_ARG);
    (void)ws_bytes;
    auto rows = [&](const kda_rows_desc* d) { return T_tot ? as_rows(d) : LatentRows{}; };
    const DecayPrefillArgs a{rows(q), rows(k), rows(v), rows(out), head_decay, log_decay, cu_seqlens,
                             init_slot, final_slot, track_chunk_idx, state_pool, track_state, dev_status, P, N, T_tot,
                             H, H / Hk, M, in_dtype, out_dtype, state_type(flags), scale};
    decay_serial_kernel<<<(unsigned)(N * H * 4), 128, 0, as_stream(stream)>>>(a);
    return launch_status();
}
