// decay_decode.cu -- kda_decay_decode: linear attention with a decay a head for 1 to 16 positions a
// request, from and to a slot-indexed state pool.
//
// K positions from a state S_0, with a_t = e^{g_t} and products of decays taken as products (no
// differences of long sums):
//     o_t = scale ( (prod_{s<=t} a_s) S_0^T q_t + sum_{j<=t} (prod_{j<s<=t} a_s) (q_t . k_j) v_j ),
//     S_n = (prod_{s<=n} a_s) S_0 + sum_{j<=n} (prod_{j<s<=n} a_s) k_j v_j^T.
// So the state is read once and, for n >= 1 committed positions, written once, however many positions
// there are: a position costs one product with the state (and one more if it is committed).
//
// Bound by HBM: the state's bytes.  A warp holds whole rows of S^T in registers (a row = one value channel,
// 128 key channels; lane l owns key channels 4l .. 4l+3), asked for at the start, so that the bytes in
// flight are the registers of all resident warps.  The row sums of a group of rows (and positions) are
// reduced together, half of them moving at each step: 31 shuffles for 32 sums in place of 160.
#include "decay_common.cuh"
#include "kda_host.h"
#include "latent_host.h"

namespace kda {
namespace {

constexpr int kDecayThreads = 128;
constexpr int kDecayMaxK = 16;

struct DecayDecodeArgs {
    LatentRows q, k, v, out;  // bases are in elements of the input (output) type
    const float *head_decay, *log_decay;
    void* pool;
    const int32_t *slot, *dst_slot, *q_len, *n_commit;
    int32_t* dev_status;
    int64_t P;
    int32_t R, K, H, group;  // group: value heads a key head
    int in_dt, out_dt;
    float scale;
};

// One request's plan: source and destination slots and how many positions there are and are committed.
struct Plan {
    int64_t src, dst;
    int ql, commit;
    bool live;
};

__device__ __forceinline__ Plan plan_of(const DecayDecodeArgs& a, int r, bool lead) {
    Plan p;
    p.src = a.slot[r];
    p.dst = a.dst_slot ? a.dst_slot[r] : p.src;
    p.ql = a.q_len ? a.q_len[r] : a.K;
    p.commit = a.n_commit ? a.n_commit[r] : p.ql;
    int bad = 0;
    if (p.src >= a.P || (p.src >= 0 && p.dst >= a.P)) bad |= KDA_DEV_BAD_SLOT;
    if (p.ql < 0 || p.ql > a.K || p.commit < 0 || p.commit > p.ql) bad |= KDA_DEV_BAD_ACCEPT;
    if (p.src < 0) bad = 0;  // a padding request: nothing of it is looked at
    p.live = p.src >= 0 && bad == 0;
    if (bad && lead) report(a.dev_status, bad);
    if (!p.live) p.ql = p.commit = 0;
    return p;
}

// Sums of N per-lane values over the warp, N = 8, 16 or 32: lane l gets the total of value l / (32 / N).
template <int N>
__device__ __forceinline__ float reduce_scatter(float (&x)[N], int lane) {
#pragma unroll
    for (int half = N / 2, off = 16; half; half >>= 1, off >>= 1) {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int e = 0; e < N / 2; ++e)
            if (e < half) {
                const float send = upper ? x[e] : x[e + half], keep = upper ? x[e + half] : x[e];
                x[e] = keep + __shfl_xor_sync(0xffffffffu, send, off);
            }
    }
    float t = x[0];
#pragma unroll
    for (int off = 16 / N; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t;
}

__device__ __forceinline__ const void* row_of(const LatentRows& d, int64_t row, int h, int dt) {
    return reinterpret_cast<const uint8_t*>(d.base) + (row * d.rs + h * d.hs) * dtype_bytes(dt);
}
__device__ __forceinline__ void* out_row(const LatentRows& d, int64_t row, int h, int dt) {
    return const_cast<void*>(row_of(d, row, h, dt));
}

// One position: 32 rows a block, eight a warp.  Nothing is shared between warps.
template <int ST>
__global__ void __launch_bounds__(kDecayThreads) decay_step_kernel(const DecayDecodeArgs a) {
    using SIO = State<ST>;
    constexpr int RW = 8, parts = kD / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / parts, part = blockIdx.x % parts;
    const int r = unit / a.H, h = unit - r * a.H;
    const Plan p = plan_of(a, r, threadIdx.x == 0 && part == 0 && h == 0);
    const int row0 = part * 32 + warp * RW;
    float4 s[RW];
    if (p.live && (p.ql || p.dst != p.src)) {
        const size_t S = state_elem(p.src, a.H, h) + (size_t)row0 * kD + 4 * lane;
#pragma unroll
        for (int i = 0; i < RW; ++i) s[i] = SIO::load4_cs(a.pool, S + (size_t)i * kD);
    }
    if (p.ql) {
        const int hk = h / a.group;
        const float4 k = load4_as(row_of(a.k, r, hk, a.in_dt), 4 * lane, a.in_dt);
        const float vm = load1_as(row_of(a.v, r, h, a.in_dt), row0 + (lane >> 2), a.in_dt);  // of the row lane / 4
        const float decay = __expf(log_decay_of(a.head_decay, a.log_decay, r, a.H, h));
        if (a.out.base) {
            float4 q = load4_as(row_of(a.q, r, hk, a.in_dt), 4 * lane, a.in_dt);
            q = make_float4(q.x * a.scale, q.y * a.scale, q.z * a.scale, q.w * a.scale);
            const float kq = warp_sum(f4_dot(k, q));
            float d[RW];
#pragma unroll
            for (int i = 0; i < RW; ++i) d[i] = f4_dot(s[i], q);
            const float o = fmaf(decay, reduce_scatter<RW>(d, lane), kq * vm);
            if ((lane & 3) == 0) store1_as(out_row(a.out, r, h, a.out_dt), row0 + (lane >> 2), o, a.out_dt);
        }
        if (p.commit) {
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const float4 x = f4_mul(s[i], make_float4(decay, decay, decay, decay));
                s[i] = f4_fma(__shfl_sync(0xffffffffu, vm, 4 * i), k, x);
            }
        }
    } else if (a.out.base) {
        if (lane < RW) store1_as(out_row(a.out, r, h, a.out_dt), row0 + lane, 0.f, a.out_dt);
    }
    if (p.live && p.dst >= 0 && (p.commit || p.dst != p.src)) {
        const size_t S = state_elem(p.dst, a.H, h) + (size_t)row0 * kD + 4 * lane;
#pragma unroll
        for (int i = 0; i < RW; ++i) SIO::store4_cs(a.pool, S + (size_t)i * kD, s[i]);
    }
}

// Several positions: 64 rows a block, sixteen a warp.  The block first leaves in shared memory the positions'
// rows, the products q_t . k_j with their decays, and each committed value with its decay.
template <int ST>
__global__ void __launch_bounds__(kDecayThreads) decay_steps_kernel(const DecayDecodeArgs a) {
    using SIO = State<ST>;
    constexpr int RW = 16, RB = 64, parts = kD / RB, K16 = kDecayMaxK;
    __shared__ __align__(16) float sq[K16][kD], sk[K16][kD], sv[K16][RB], fv[K16][RB];
    __shared__ float w[K16][K16], lead[K16], dec[K16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / parts, part = blockIdx.x % parts;
    const int r = unit / a.H, h = unit - r * a.H, hk = h / a.group;
    const Plan p = plan_of(a, r, threadIdx.x == 0 && part == 0 && h == 0);
    const int ql = p.ql, nc = p.commit, row0 = warp * RW;
    const bool answer = a.out.base != nullptr;
    const bool moved = p.live && p.dst >= 0 && p.dst != p.src;
    float4 s[RW];
    if ((ql && answer) || nc || moved) {
        const size_t S = state_elem(p.src, a.H, h) + (size_t)(part * RB + row0) * kD + 4 * lane;
#pragma unroll
        for (int i = 0; i < RW; ++i) s[i] = SIO::load4_cs(a.pool, S + (size_t)i * kD);
    }
    const int64_t first = (int64_t)r * a.K;
    for (int t = ql + warp; answer && t < a.K; t += 4)  // positions that there are not
        for (int i = lane; i < RB; i += 32) store1_as(out_row(a.out, first + t, h, a.out_dt), part * RB + i, 0.f, a.out_dt);
    if (ql) {
        if (threadIdx.x < ql) dec[threadIdx.x] = __expf(log_decay_of(a.head_decay, a.log_decay, first + threadIdx.x, a.H, h));
        for (int t = warp; t < ql; t += 4) {
            if (answer) {
                const float4 q = load4_as(row_of(a.q, first + t, hk, a.in_dt), 4 * lane, a.in_dt);
                *reinterpret_cast<float4*>(&sq[t][4 * lane]) = make_float4(q.x * a.scale, q.y * a.scale, q.z * a.scale, q.w * a.scale);
            }
            *reinterpret_cast<float4*>(&sk[t][4 * lane]) = load4_as(row_of(a.k, first + t, hk, a.in_dt), 4 * lane, a.in_dt);
            if (lane < RB / 4)
                *reinterpret_cast<float4*>(&sv[t][4 * lane]) =
                    load4_as(row_of(a.v, first + t, h, a.in_dt), part * RB + 4 * lane, a.in_dt);
        }
        __syncthreads();
        // thread j: prod_{j<s<=t} a_s for t >= j, and of the committed ones the factor of v_j
        if (threadIdx.x < ql) {
            const int j = threadIdx.x;
            float f = 1.f;
            w[j][j] = 1.f;
            for (int t = j + 1; t < ql; ++t) w[t][j] = f *= dec[t];
            f = 1.f;
            for (int t = 0; t <= j; ++t) f *= dec[t];
            lead[j] = f;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < nc * RB; e += kDecayThreads) {
            const int j = e / RB, i = e % RB;
            fv[j][i] = w[nc - 1][j] * sv[j][i];
        }
        __syncthreads();
        if (answer) {
            // products with the keys, 32 pairs (t, j) of a warp together
            for (int base = warp * 32; base < ql * ql; base += 128) {
                float d[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const int pair = min(base + e, ql * ql - 1), t = pair / ql, j = pair - t * ql;
                    d[e] = f4_dot(*reinterpret_cast<const float4*>(&sq[t][4 * lane]), *reinterpret_cast<const float4*>(&sk[j][4 * lane]));
                }
                const float x = reduce_scatter<32>(d, lane);
                const int pair = base + lane, t = pair / ql, j = pair - t * ql;
                if (pair < ql * ql && j <= t) w[t][j] *= x;
            }
            __syncthreads();
            for (int t0 = 0; t0 < ql; t0 += 2) {  // two positions of sixteen rows: 32 sums
                float d[32];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float4 q = *reinterpret_cast<const float4*>(&sq[min(t0 + u, ql - 1)][4 * lane]);
#pragma unroll
                    for (int i = 0; i < RW; ++i) d[16 * u + i] = f4_dot(s[i], q);
                }
                const float x = reduce_scatter<32>(d, lane);
                const int t = t0 + (lane >> 4), i = row0 + (lane & 15);
                if (t < ql) {
                    float o = lead[t] * x;
                    for (int j = 0; j <= t; ++j) o = fmaf(w[t][j], sv[j][i], o);
                    store1_as(out_row(a.out, first + t, h, a.out_dt), part * RB + i, o, a.out_dt);
                }
            }
        }
        if (nc) {
            const float f = lead[nc - 1];
#pragma unroll
            for (int i = 0; i < RW; ++i) s[i] = f4_mul(s[i], make_float4(f, f, f, f));
            for (int j = 0; j < nc; ++j) {
                const float4 k = *reinterpret_cast<const float4*>(&sk[j][4 * lane]);
#pragma unroll
                for (int i = 0; i < RW; i += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(&fv[j][row0 + i]);
                    s[i] = f4_fma(v.x, k, s[i]);
                    s[i + 1] = f4_fma(v.y, k, s[i + 1]);
                    s[i + 2] = f4_fma(v.z, k, s[i + 2]);
                    s[i + 3] = f4_fma(v.w, k, s[i + 3]);
                }
            }
        }
    }
    if (p.live && p.dst >= 0 && (nc || moved)) {
        const size_t S = state_elem(p.dst, a.H, h) + (size_t)(part * RB + row0) * kD + 4 * lane;
#pragma unroll
        for (int i = 0; i < RW; ++i) SIO::store4_cs(a.pool, S + (size_t)i * kD, s[i]);
    }
}

template <int ST>
void launch(const DecayDecodeArgs& a, cudaStream_t s) {
    const unsigned units = (unsigned)a.R * (unsigned)a.H;
    if (a.K == 1)
        decay_step_kernel<ST><<<units * 4, kDecayThreads, 0, s>>>(a);
    else
        decay_steps_kernel<ST><<<units * 2, kDecayThreads, 0, s>>>(a);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_decay_decode(const kda_rows_desc* q, const kda_rows_desc* k, const kda_rows_desc* v,
                                       kda_dtype in_dtype, const float* head_decay, const float* log_decay, int32_t R,
                                       int32_t K, const int32_t* q_len, const int32_t* n_commit, int32_t H, int32_t Hk,
                                       int32_t dk, int32_t dv, float scale, uint32_t flags, void* state_pool, int64_t P,
                                       const int32_t* slot, const int32_t* dst_slot, const kda_rows_desc* out,
                                       kda_dtype out_dtype, int32_t* dev_status, void* stream) {
    KDA_REQUIRE(R >= 0 && K >= 0 && H > 0 && Hk > 0 && P >= 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(H % Hk == 0 && isfinite(scale), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(dk == kD && dv == kD && K <= kDecayMaxK, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(any_dtype_ok(in_dtype) && any_dtype_ok(out_dtype), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((flags & ~(KDA_STATE_BF16 | KDA_STATE_F16)) == 0 && state_flags_ok(flags), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((int64_t)R * H * 4 < (1ll << 31) && (int64_t)R * K < (1ll << 31), KDA_ERR_UNSUPPORTED);
    if (R == 0 || K == 0) return KDA_OK;
    KDA_REQUIRE(rows_ok(k) && rows_ok(v) && (!out || (rows_ok(out) && rows_ok(q))), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(head_decay || log_decay, KDA_ERR_INVALID_ARG);
    const void* need[] = {state_pool, slot};
    for (const void* p : need) KDA_REQUIRE(p != nullptr, KDA_ERR_INVALID_ARG);
    const void* ptrs[] = {state_pool, slot, dst_slot, q_len, n_commit, head_decay, log_decay};
    for (const void* p : ptrs) KDA_REQUIRE(aligned16(p), KDA_ERR_INVALID_ARG);
    DecayDecodeArgs a{};
    a.k = as_rows(k);
    a.v = as_rows(v);
    if (out) a.q = as_rows(q), a.out = as_rows(out);
    a.head_decay = head_decay;
    a.log_decay = log_decay;
    a.pool = state_pool;
    a.slot = slot;
    a.dst_slot = dst_slot;
    a.q_len = q_len;
    a.n_commit = n_commit;
    a.dev_status = dev_status;
    a.P = P;
    a.R = R;
    a.K = K;
    a.H = H;
    a.group = H / Hk;
    a.in_dt = in_dtype;
    a.out_dt = out_dtype;
    a.scale = scale;
    switch (state_type(flags)) {
        case kStateBF16: launch<kStateBF16>(a, as_stream(stream)); break;
        case kStateF16: launch<kStateF16>(a, as_stream(stream)); break;
        default: launch<kStateF32>(a, as_stream(stream));
    }
    return launch_status();
}
