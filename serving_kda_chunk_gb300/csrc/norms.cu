// norms.cu -- kda_gated_norm and kda_residual_norm: the row norms around a block, with the gate and
// the residual sum that stand beside them.
//
//   gated:     y = x / sqrt(mean(x^2) + eps) (w + offset) act(gate)      (per row and head)
//   residual:  z = post ? x / sqrt(mean(x^2) + eps) (post + offset) : x
//              h = residual_scale r + branch_scale act(gate) z
//              y = h / sqrt(mean(h^2) + eps) (w + offset)                (per row)
//
// One pass: a row lives in the registers of the TPR threads that share it (NV vectors of eight elements
// each), so every input is read once and every output written once, and the second norm of the residual
// form costs a reduction and no traffic.  Bound by HBM.  All arithmetic is fp32; y comes from the
// unrounded h, and each output is rounded once on its store.  41460 rows, bf16: gated, 32 heads of 128, 148 us (the
// measured copy rate); residual of 4096 channels 215 us (94 % of it).
#include "kda_host.h"
#include "latent_common.cuh"
#include "umma.cuh"

#include <initializer_list>

namespace kda {
namespace {

constexpr int kNormMaxDim = 16384;
constexpr int kStreamStages = 8, kStreamBytes = 210 * 1024;  // most rows in a block's ring; bytes of a SM's rings

struct NormRows {
    const void* base;
    int64_t rs, hs;  // strides of rows and heads, in elements
};

// The element a thread holds as (vector i, element e): eight neighbours when rows are whole 16-byte
// vectors, else neighbours lie in neighbouring threads so that single loads are side by side.
template <bool kVec, int TPR>
__device__ __forceinline__ int elem_at(int i, int e, int t) {
    return kVec ? (i * TPR + t) * 8 + e : (i * 8 + e) * TPR + t;
}

// Raw bits of eight elements: what a load leaves in registers until it is used.
template <int DT>
struct Raw8 {
    uint32_t w[DT == KDA_F32 ? 8 : 4];
};

template <int DT, bool kVec, int TPR>
__device__ __forceinline__ Raw8<DT> load_raw(const void* row, int i, int t, int d) {
    Raw8<DT> r;
    if constexpr (kVec) {
        const int at = elem_at<true, TPR>(i, 0, t);
        const uint4 zero = make_uint4(0, 0, 0, 0);
        if constexpr (DT == KDA_F32) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + at);
            const uint4 a = at < d ? p[0] : zero, b = at < d ? p[1] : zero;
            r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
            r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
        } else {
            const uint4 a = at < d ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + at) : zero;
            r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        }
    } else {
        if constexpr (DT == KDA_F32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = elem_at<false, TPR>(i, e, t);
                r.w[e] = at < d ? static_cast<const uint32_t*>(row)[at] : 0u;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const int a = elem_at<false, TPR>(i, e, t), b = elem_at<false, TPR>(i, e + 1, t);
                const uint32_t lo = a < d ? static_cast<const uint16_t*>(row)[a] : 0;
                const uint32_t hi = b < d ? static_cast<const uint16_t*>(row)[b] : 0;
                r.w[e / 2] = lo | hi << 16;
            }
        }
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void widen(const Raw8<DT>& r, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (DT == KDA_F32) {
            v[2 * e] = __uint_as_float(r.w[2 * e]);
            v[2 * e + 1] = __uint_as_float(r.w[2 * e + 1]);
        } else {
            const float2 f = Elem<DT>::get2(r.w[e]);
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
        }
    }
}

template <int DT, bool kVec, int TPR>
__device__ __forceinline__ void store8(void* row, int i, int t, int d, const float (&v)[8]) {
    if constexpr (kVec) {
        const int at = elem_at<true, TPR>(i, 0, t);
        if (at >= d) return;
        if constexpr (DT == KDA_F32) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + at);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + at) =
                make_uint4(Elem<DT>::put2(v[0], v[1]), Elem<DT>::put2(v[2], v[3]), Elem<DT>::put2(v[4], v[5]),
                           Elem<DT>::put2(v[6], v[7]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int at = elem_at<false, TPR>(i, e, t);
            if (at >= d) continue;
            if constexpr (DT == KDA_F32)
                static_cast<float*>(row)[at] = v[e];
            else
                static_cast<uint16_t*>(row)[at] = (uint16_t)Elem<DT>::put2(v[e], 0.f);
        }
    }
}

template <bool kVec, int TPR>
__device__ __forceinline__ void store8_as(void* row, int i, int t, int d, const float (&v)[8], int dt) {
    if (dt == KDA_F32) store8<KDA_F32, kVec, TPR>(row, i, t, d, v);
    else if (dt == KDA_BF16) store8<KDA_BF16, kVec, TPR>(row, i, t, d, v);
    else store8<KDA_F16, kVec, TPR>(row, i, t, d, v);
}

__device__ __forceinline__ void* at_elem(void* p, int64_t i, int dt) {
    return static_cast<uint8_t*>(p) + i * dtype_bytes(dt);
}
__device__ __forceinline__ const void* at_elem(const void* p, int64_t i, int dt) {
    return static_cast<const uint8_t*>(p) + i * dtype_bytes(dt);
}

// Sum over the TPR threads of a row: within a warp, or over the block, which then holds one row.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* part) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) x += part[w];
    }
    return x;
}

// act(z) of two values; e^-z = inf gives 0 (z = -inf gives silu NaN, as -inf * 0 does).  One exponential and one
// reciprocal a value, both the fast ones (2^-22).
template <int ACT>
__device__ __forceinline__ float2 act2(float2 z) {
    if constexpr (ACT == KDA_ACT_NONE) return z;
    const float2 e = __fmul2_rn(z, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    const float2 d = __fadd2_rn(make_float2(ex2(e.x), ex2(e.y)), make_float2(1.f, 1.f));
    const float2 s = make_float2(__fdividef(1.f, d.x), __fdividef(1.f, d.y));
    return ACT == KDA_ACT_SILU ? __fmul2_rn(z, s) : s;
}
// Runs body(ACT) with the activation fixed at compile time: tested at each element it cost a branch there.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& body) {
    if (act == KDA_ACT_SILU) body(std::integral_constant<int, KDA_ACT_SILU>{});
    else if (act == KDA_ACT_SIGMOID) body(std::integral_constant<int, KDA_ACT_SIGMOID>{});
    else body(std::integral_constant<int, KDA_ACT_NONE>{});
}

// Pairs of a vector of eight.
__device__ __forceinline__ float2 pair(const float (&v)[8], int e) { return make_float2(v[2 * e], v[2 * e + 1]); }
__device__ __forceinline__ void set_pair(float (&v)[8], int e, float2 x) { v[2 * e] = x.x, v[2 * e + 1] = x.y; }

template <int NV>
__device__ __forceinline__ float sum_sq(const float (&v)[NV][8]) {
    float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e & 1] = __ffma2_rn(pair(v[i], e), pair(v[i], e), s[e & 1]);
    return (s[0].x + s[0].y) + (s[1].x + s[1].y);
}

constexpr int norm_threads(int tpr) { return tpr > 256 ? tpr : tpr > 32 ? tpr : 256; }

// U rows a thread group at a time: their loads are in flight together.
template <int DT, bool kVec, int TPR, int NV, int U>
__global__ void __launch_bounds__(norm_threads(TPR)) gated_norm_kernel(
    NormRows x, NormRows gate, const void* __restrict__ weight, int64_t n, int H, int d, float inv_d, float eps,
    float offset, int act, bool gate_first, NormRows out, int out_dt) {
    __shared__ float part[TPR > 32 ? TPR / 32 : 1];
    constexpr int G = norm_threads(TPR) / TPR;  // rows a block at a time
    const int t = threadIdx.x % TPR;
    const int64_t first = (int64_t)blockIdx.x * (G * U) + threadIdx.x / TPR;
    // rows that lie evenly come as heads of one row each (H = 1): no division
    auto place = [&](const NormRows& at, int64_t row) {
        if (H == 1) return row * at.rs;
        const int64_t r = row / H;
        return r * at.rs + (row - r * H) * at.hs;
    };
    Raw8<DT> xr[U][NV], gr[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = first + u * G;
        const int dd = row < n ? d : 0;  // a row past the end loads and stores nothing
        const void* xp = at_elem(x.base, place(x, row), DT);
#pragma unroll
        for (int i = 0; i < NV; ++i) xr[u][i] = load_raw<DT, kVec, TPR>(xp, i, t, dd);
        if (gate.base) {
            const void* gp = at_elem(gate.base, place(gate, row), DT);
#pragma unroll
            for (int i = 0; i < NV; ++i) gr[u][i] = load_raw<DT, kVec, TPR>(gp, i, t, dd);
        }
    }
    float w[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (weight) widen<DT>(load_raw<DT, kVec, TPR>(weight, i, t, d), w[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i][e] = weight ? w[i][e] + offset : 1.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = first + u * G;
        const int dd = row < n ? d : 0;
        float v[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) widen<DT>(xr[u][i], v[i]);
        auto times_gate = [&](bool mask) {
            with_act(act, [&](auto ACT) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float g[8];
                    widen<DT>(gr[u][i], g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) set_pair(v[i], e, __fmul2_rn(pair(v[i], e), act2<ACT>(pair(g, e))));
                    // an absent element counts as zero, whatever act(0) makes of it
                    if (mask)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (elem_at<kVec, TPR>(i, e, t) >= dd) v[i][e] = 0.f;
                }
            });
        };
        if (gate.base && gate_first) times_gate(true);
        const float f = rsqrtf(row_sum<TPR>(sum_sq<NV>(v), part) * inv_d + eps);
        if (gate.base && !gate_first) times_gate(false);
        void* to = at_elem(const_cast<void*>(out.base), place(out, row), out_dt);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) set_pair(v[i], e, __fmul2_rn(__fmul2_rn(pair(v[i], e), make_float2(f, f)), pair(w[i], e)));
            store8_as<kVec, TPR>(to, i, t, dd, v[i], out_dt);
        }
        if (TPR > 32 && U > 1) __syncthreads();  // part is written again
    }
}

struct ResidualArgs {
    const void *x, *residual, *post, *gate, *weight;
    void *hidden, *out;
    int64_t xs, rs, gs, hs, os;  // row strides, in elements
    int64_t n;
    int d, act, res_dt, out_dt;
    float inv_d, rscale, bscale, eps, offset;
};

template <int DT, bool kVec, int TPR, int NV>
__global__ void __launch_bounds__(norm_threads(TPR)) residual_norm_kernel(const ResidualArgs a) {
    __shared__ float part[2][TPR > 32 ? TPR / 32 : 1];
    constexpr int G = norm_threads(TPR) / TPR;
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * G + threadIdx.x / TPR;
    const int d = row < a.n ? a.d : 0;
    Raw8<DT> xr[NV], gr[NV], pr[NV], wr[NV];
    float r[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) xr[i] = load_raw<DT, kVec, TPR>(at_elem(a.x, row * a.xs, DT), i, t, d);
    if (a.res_dt == KDA_F32) {
#pragma unroll
        for (int i = 0; i < NV; ++i) widen<KDA_F32>(load_raw<KDA_F32, kVec, TPR>(at_elem(a.residual, row * a.rs, KDA_F32), i, t, d), r[i]);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) widen<DT>(load_raw<DT, kVec, TPR>(at_elem(a.residual, row * a.rs, DT), i, t, d), r[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (a.gate) gr[i] = load_raw<DT, kVec, TPR>(at_elem(a.gate, row * a.gs, DT), i, t, d);
        if (a.post) pr[i] = load_raw<DT, kVec, TPR>(a.post, i, t, d);
        if (a.weight) wr[i] = load_raw<DT, kVec, TPR>(a.weight, i, t, d);
    }
    float z[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) widen<DT>(xr[i], z[i]);
    float f = a.bscale;
    if (a.post) f *= rsqrtf(row_sum<TPR>(sum_sq<NV>(z), part[0]) * a.inv_d + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float p[8], g[8];
        if (a.post) widen<DT>(pr[i], p);
        if (a.gate) {
            widen<DT>(gr[i], g);
            with_act(a.act, [&](auto ACT) {
#pragma unroll
                for (int e = 0; e < 4; ++e) set_pair(g, e, act2<ACT>(pair(g, e)));
            });
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float y = z[i][e] * f;
            if (a.post) y *= p[e] + a.offset;
            if (a.gate) y *= g[e];
            z[i][e] = fmaf(a.rscale, r[i][e], y);
            // an absent element counts as zero, whatever act(0) and the offset make of it
            if (elem_at<kVec, TPR>(i, e, t) >= d) z[i][e] = 0.f;
        }
    }
    if (a.hidden) {
        void* p = at_elem(a.hidden, row * a.hs, a.res_dt);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (a.res_dt == KDA_F32) store8<KDA_F32, kVec, TPR>(p, i, t, d, z[i]);
            else store8<DT, kVec, TPR>(p, i, t, d, z[i]);
        }
    }
    if (!a.out) return;
    f = rsqrtf(row_sum<TPR>(sum_sq<NV>(z), part[1]) * a.inv_d + a.eps);
    void* p = at_elem(a.out, row * a.os, a.out_dt);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float w[8];
        if (a.weight) widen<DT>(wr[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[i][e] *= a.weight ? f * (w[e] + a.offset) : f;
        store8_as<kVec, TPR>(p, i, t, d, z[i], a.out_dt);
    }
}

// Many long rows: a block walks rows gridDim.x apart, and a ring of rows in shared memory, filled by bulk copies,
// keeps HBM busy under the two reductions and the stores.  (Rows in registers alone, 128 threads of four vectors:
// 140 registers, 17 % of the warps and 4.5 of 6.7 TB/s at 41460 x 4096.)
template <int T, int NV>
constexpr int stream_ctas = T == 128 ? 4 : T == 256 ? (NV == 1 ? 3 : 2) : (NV <= 2 ? 2 : 1);  // blocks a SM, by registers

template <int DT, int RDT, int T, int NV>
__global__ void __launch_bounds__(T, stream_ctas<T, NV>) residual_stream_kernel(const ResidualArgs a, int stages) {
    using namespace umma;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t full[kStreamStages];
    __shared__ float part[2][2][T / 32];  // two sums, of even and odd rows: one barrier lies between two uses
    __shared__ int gone;
    const int t = threadIdx.x, d = a.d, xb = d * dtype_bytes(DT), rb = d * dtype_bytes(RDT);
    const bool gates = a.gate && a.gs != 0;  // a gate row a row
    const int stage_bytes = xb + rb + (gates ? xb : 0);
    if (t == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&full[i]), 1);
        gone = 0;
    }
    __syncthreads();
    auto ask = [&](int64_t row, int st) {  // by thread 0
        const uint32_t bar = smem_u32(&full[st]), to = smem_u32(ring) + st * stage_bytes;
        mbar_expect_tx(bar, stage_bytes);
        bulk_load(to, at_elem(a.x, row * a.xs, DT), xb, bar);
        bulk_load(to + xb, at_elem(a.residual, row * a.rs, RDT), rb, bar);
        if (gates) bulk_load(to + xb + rb, at_elem(a.gate, row * a.gs, DT), xb, bar);
    };
    if (t == 0)
        for (int i = 0; i < stages; ++i)
            if (blockIdx.x + (int64_t)i * gridDim.x < a.n) ask(blockIdx.x + (int64_t)i * gridDim.x, i);
    // What multiplies each channel of the branch (post weight, a gate shared by the rows, the branch's scale) and of
    // the output, made once: in registers, or where a thread has more than two vectors anew for each row.
    auto factors = [&](int i, float (&before)[8], float (&after)[8]) {
        float y[8];
        if (a.post) {
            widen<DT>(load_raw<DT, true, T>(a.post, i, t, d), before);
#pragma unroll
            for (int e = 0; e < 8; ++e) before[e] = (before[e] + a.offset) * a.bscale;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) before[e] = a.bscale;
        }
        if (a.gate && !gates) {
            widen<DT>(load_raw<DT, true, T>(a.gate, i, t, d), y);
            with_act(a.act, [&](auto ACT) {
#pragma unroll
                for (int e = 0; e < 4; ++e) set_pair(before, e, __fmul2_rn(pair(before, e), act2<ACT>(pair(y, e))));
            });
        }
        if (a.weight) widen<DT>(load_raw<DT, true, T>(a.weight, i, t, d), after);
#pragma unroll
        for (int e = 0; e < 8; ++e) after[e] = a.weight ? after[e] + a.offset : 1.f;
    };
    constexpr bool kKeep = NV <= 2;
    float before[kKeep ? NV : 1][8], after[kKeep ? NV : 1][8];
    if constexpr (kKeep)
#pragma unroll
        for (int i = 0; i < NV; ++i) factors(i, before[i], after[i]);
    uint32_t it = 0;
    bool lost = false;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, ++it) {
        const int st = it % stages;
        // (a copy that does not come within about a second: NaN for the block's rows from there on)
        if (!lost && !mbar_wait(smem_u32(&full[st]), (it / stages) & 1, 1u << 18)) gone = 1;
        const uint8_t* xs = ring + st * stage_bytes;
        float z[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) widen<DT>(load_raw<DT, true, T>(xs, i, t, d), z[i]);
        float f = 1.f;
        if (a.post) f = rsqrtf(row_sum<T>(sum_sq<NV>(z), part[0][it & 1]) * a.inv_d + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (elem_at<true, T>(i, 0, t) >= d) continue;  // (zeros, which add nothing)
            float y[8];
            if constexpr (!kKeep) factors(i, before[0], after[0]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                set_pair(z[i], e, __fmul2_rn(__fmul2_rn(pair(z[i], e), make_float2(f, f)), pair(before[kKeep ? i : 0], e)));
            if (gates) {
                widen<DT>(load_raw<DT, true, T>(xs + xb + rb, i, t, d), y);
                with_act(a.act, [&](auto ACT) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) set_pair(z[i], e, __fmul2_rn(pair(z[i], e), act2<ACT>(pair(y, e))));
                });
            }
            widen<RDT>(load_raw<RDT, true, T>(xs + xb, i, t, d), y);
#pragma unroll
            for (int e = 0; e < 4; ++e) set_pair(z[i], e, __ffma2_rn(make_float2(a.rscale, a.rscale), pair(y, e), pair(z[i], e)));
        }
        float sum = row_sum<T>(sum_sq<NV>(z), part[1][it & 1]);
        // all have read the row (and the mark): the next one may come over it
        lost = gone;
        if (lost) {
            sum = __int_as_float(0x7fc00000);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) z[i][e] = sum;
        } else if (t == 0 && row + (int64_t)stages * gridDim.x < a.n) {
            ask(row + (int64_t)stages * gridDim.x, st);
        }
        if (a.hidden) {
            void* p = at_elem(a.hidden, row * a.hs, RDT);
#pragma unroll
            for (int i = 0; i < NV; ++i) store8<RDT, true, T>(p, i, t, d, z[i]);
        }
        if (a.out) {
            f = rsqrtf(sum * a.inv_d + a.eps);
            void* p = at_elem(a.out, row * a.os, a.out_dt);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if constexpr (!kKeep) factors(i, before[0], after[0]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    set_pair(z[i], e, __fmul2_rn(__fmul2_rn(pair(z[i], e), make_float2(f, f)), pair(after[kKeep ? i : 0], e)));
                store8_as<true, T>(p, i, t, d, z[i], a.out_dt);
            }
        }
    }
    if (lost && t == 0)  // copies in flight land before the block's memory goes
        for (int i = 0; i < 1000; ++i) __nanosleep(1000000);
}

inline bool dtype_known(kda_dtype d) { return d == KDA_BF16 || d == KDA_F16 || d == KDA_F32; }
inline bool elem_aligned(const void* p, kda_dtype dt) { return reinterpret_cast<uintptr_t>(p) % dtype_bytes(dt) == 0; }
// Whole 16-byte vectors of eight elements: the row length, and each tensor's start and strides.
inline bool vec_ok(const void* p, int64_t rs, int64_t hs) { return p == nullptr || (aligned16(p) && rs % 8 == 0 && hs % 8 == 0); }

// Calls launch(TPR, NV) for the form that holds a row of nvec vectors: one vector a thread as long as a block of 256
// takes the row, at any number of rows (residual, bf16, 16384 rows of 1024: 29 us, and 40 with four vectors a thread of a
// warp; 512: 16 and 36).  Longer rows of whole vectors: 512 threads while there are fewer rows than fill the device (`few`;
// 4096 channels, gated: 64 rows 2.4 and 2.8 us, 1024 rows 8.9 and 9.2), else four vectors a thread, which keep more
// bytes in flight and share the reductions (8192 rows 39 and 45); above 512 vectors two a thread (8192 channels, residual,
// 200 rows: 5.6 us, 1024 x 1 6.3, 512 x 4 7.4), above 1024 four (11.0; 1024 x 2 12.6).  Rows of single elements, whose
// accesses are eight times as many, want every thread (8192 rows, residual: 4095 channels 102 us, 128 x 4 110; 4097
// 211, 512 x 4 329).
template <bool kVec, class F>
void with_row_form(int nvec, bool few, F&& launch) {
    if (nvec <= 8) launch(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
    else if (nvec <= 16) launch(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    else if (nvec <= 32) launch(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
    else if (nvec <= 64) launch(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    else if (nvec <= 128) launch(std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
    else if (nvec <= 256) launch(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    else if (nvec <= 512 && (few || !kVec)) launch(std::integral_constant<int, 512>{}, std::integral_constant<int, 1>{});
    else if constexpr (!kVec) {
        if (nvec <= 1024) launch(std::integral_constant<int, 1024>{}, std::integral_constant<int, 1>{});
        else launch(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
    } else if (nvec <= 512) launch(std::integral_constant<int, 128>{}, std::integral_constant<int, 4>{});
    else if (nvec <= 1024) launch(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
    else launch(std::integral_constant<int, 512>{}, std::integral_constant<int, 4>{});
}

template <class F>
void with_types(kda_dtype dt, bool vec, F&& f) {
    auto by_vec = [&](auto DT) {
        if (vec) f(DT, std::true_type{});
        else f(DT, std::false_type{});
    };
    if (dt == KDA_BF16) by_vec(std::integral_constant<int, KDA_BF16>{});
    else if (dt == KDA_F16) by_vec(std::integral_constant<int, KDA_F16>{});
    else by_vec(std::integral_constant<int, KDA_F32>{});
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_gated_norm(const kda_rows_desc* x, const kda_rows_desc* gate, const void* weight,
                                     kda_dtype in_dtype, int32_t R, int32_t H, int32_t d, float eps,
                                     float weight_offset, kda_act act, uint32_t flags, const kda_rows_desc* out,
                                     kda_dtype out_dtype, void* stream) {
    KDA_REQUIRE(R >= 0 && H > 0 && d > 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(dtype_known(in_dtype) && dtype_known(out_dtype) && d <= kNormMaxDim, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(act >= KDA_ACT_NONE && act <= KDA_ACT_SILU && (flags & ~KDA_NORM_AFTER_GATE) == 0, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(isfinite(eps) && eps >= 0.f && isfinite(weight_offset), KDA_ERR_INVALID_ARG);
    if (R == 0) return KDA_OK;
    KDA_REQUIRE(x && out && x->base && out->base && (!gate || gate->base), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(elem_aligned(x->base, in_dtype) && elem_aligned(out->base, out_dtype), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE((!gate || elem_aligned(gate->base, in_dtype)) && elem_aligned(weight, in_dtype), KDA_ERR_INVALID_ARG);
    const NormRows xd{x->base, x->row_stride, x->head_stride}, od{out->base, out->row_stride, out->head_stride};
    const NormRows gd = gate ? NormRows{gate->base, gate->row_stride, gate->head_stride} : NormRows{nullptr, 0, 0};
    const bool vec = d % 8 == 0 && vec_ok(xd.base, xd.rs, xd.hs) && vec_ok(od.base, od.rs, od.hs) &&
                     vec_ok(gd.base, gd.rs, gd.hs) && vec_ok(weight, 0, 0);
    const int64_t n = (int64_t)R * H;
    // rows and heads that lie evenly are rows alone
    auto even = [&](NormRows& t) { return t.base == nullptr || H == 1 || R == 1 || t.rs == H * t.hs; };
    NormRows xe = xd, ge = gd, oe = od;
    const bool flat = even(xe) && even(ge) && even(oe);
    if (flat)
        for (NormRows* t : {&xe, &ge, &oe})
            if (H > 1) t->rs = t->hs;
    const int heads = flat ? 1 : H;
    const int nvec = (d + 7) / 8;
    cudaStream_t s = as_stream(stream);
    bool fits = true;
    with_types(in_dtype, vec, [&](auto DT, auto V) {
        with_row_form<V>(nvec, n < 1024, [&](auto TPR, auto NV) {
            auto run = [&](auto U) {
                constexpr int rows = norm_threads(TPR) / TPR * U;
                const int64_t blocks = (n + rows - 1) / rows;
                fits = blocks < (1ll << 31);
                if (fits)
                    gated_norm_kernel<DT, V, TPR, NV, U><<<(unsigned)blocks, norm_threads(TPR), 0, s>>>(
                        xe, ge, weight, n, heads, d, 1.f / (float)d, eps, weight_offset, act,
                        (flags & KDA_NORM_AFTER_GATE) != 0, oe, out_dtype);
            };
            // rows of one vector a thread of a warp go four at a time when there are many (128 channels: 131072 rows 20.2 and
            // 21.1 us, 524288 rows 62 and 74; 65536 rows 12.6 and 12.3, 8192 rows 3.5 and 2.6)
            if constexpr (NV == 1 && TPR <= 32) {
                if (n >= 131072) run(std::integral_constant<int, 4>{});
                else run(std::integral_constant<int, 1>{});
            } else {
                run(std::integral_constant<int, 1>{});
            }
        });
    });
    return fits ? launch_status() : KDA_ERR_UNSUPPORTED;
}

extern "C" kda_status kda_residual_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                        kda_dtype residual_dtype, const void* post_weight, const void* gate,
                                        int64_t gate_stride, kda_act act, const void* weight, kda_dtype in_dtype,
                                        int32_t R, int32_t d, float residual_scale, float branch_scale, float eps,
                                        float weight_offset, void* hidden, int64_t hidden_stride, void* out,
                                        int64_t out_stride, kda_dtype out_dtype, void* stream) {
    KDA_REQUIRE(R >= 0 && d > 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(dtype_known(in_dtype) && dtype_known(out_dtype) && d <= kNormMaxDim, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(residual_dtype == in_dtype || residual_dtype == KDA_F32, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(act >= KDA_ACT_NONE && act <= KDA_ACT_SILU, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(isfinite(eps) && eps >= 0.f && isfinite(weight_offset), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(isfinite(residual_scale) && isfinite(branch_scale), KDA_ERR_INVALID_ARG);
    if (R == 0) return KDA_OK;
    KDA_REQUIRE(x && residual && (hidden || out), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(elem_aligned(x, in_dtype) && elem_aligned(residual, residual_dtype) && elem_aligned(hidden, residual_dtype) &&
                    elem_aligned(out, out_dtype) && elem_aligned(gate, in_dtype) && elem_aligned(weight, in_dtype) &&
                    elem_aligned(post_weight, in_dtype),
                KDA_ERR_INVALID_ARG);
    const bool vec = d % 8 == 0 && vec_ok(x, x_stride, 0) && vec_ok(residual, residual_stride, 0) &&
                     vec_ok(hidden, hidden_stride, 0) && vec_ok(out, out_stride, 0) && vec_ok(gate, gate_stride, 0) &&
                     vec_ok(weight, 0, 0) && vec_ok(post_weight, 0, 0);
    const ResidualArgs a{x, residual, post_weight, gate, weight, hidden, out, x_stride, residual_stride, gate_stride,
                         hidden_stride, out_stride, R, d, act, residual_dtype, out_dtype, 1.f / (float)d, residual_scale,
                         branch_scale, eps, weight_offset};
    cudaStream_t s = as_stream(stream);
    const int stage = d * (dtype_bytes(in_dtype) * (gate && gate_stride != 0 ? 2 : 1) + dtype_bytes(residual_dtype));
    // The ring above 1024 channels, from 1024 rows on (against rows in registers: bf16, 1032 channels 84 and 137 us at 41460
    // rows, 10.2 and 13.4 at 4096, 4.4 and 4.5 at 1024, with an fp32 residual 107 and 140, 13.4 and 15.4, but 5.1 and 4.4; 4096
    // channels 25 and 33 at 4096 rows, 10.3 and 11.9 at 1024; fp32 residual 37 and 41, 13.9 and 14.6; but 1024 channels 14 and
    // 10 at 4096 rows), and above 4096 channels from 256 rows on (8192 channels: 6.1 and 8.6, 15.8 and 28 at 1024).
    if (vec && d > 1024 && R >= (d > 4096 ? 256 : 1024) && 2 * stage <= kStreamBytes) {
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return runtime_failed();
        cudaError_t err = cudaSuccess;
        auto run = [&](auto DT, auto RDT, auto T, auto NV) {
            constexpr int most = stream_ctas<T, NV>;
            const int ctas = most * 2 * stage <= kStreamBytes ? most : kStreamBytes / (2 * stage);
            const int fit = kStreamBytes / (ctas * stage), stages = fit < kStreamStages ? fit : kStreamStages;
            auto* f = residual_stream_kernel<DT, RDT, T, NV>;
            err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamBytes);
            if (err == cudaSuccess) f<<<(unsigned)(sms * ctas < R ? sms * ctas : R), T(), stages * stage, s>>>(a, stages);
        };
        auto by_len = [&](auto DT, auto RDT) {
            // Threads and vectors of each: by how many threads a row leaves idle, and how many rows a SM then has.  bf16: 1280
            // channels, 41460 rows 84 us (256 x 1: 105), but with an fp32 residual 118 and 109; 3584 channels, 16384 rows 74
            // (512 x 1: 88); 5120, 16384 rows 127 (256 x 4: 168); 16384 channels 429 (256 x 8: 847).  512 x 1 against 256 x 2 at
            // 4096 channels: 8192 rows 47.5 and 45.8, 16384 rows 88 and 94, 24000 126 and 139, 41460 211 and 237; 3976 channels
            // 47 and 44, 88 and 85, 125 and 129, 212 and 223; with an fp32 residual 144 and 137 at 16384 x 4096, 351 and 348 at
            // 41460, though 124 and 134 at 16384 x 3976: there it is left.
            using T128 = std::integral_constant<int, 128>;
            using T256 = std::integral_constant<int, 256>;
            using T512 = std::integral_constant<int, 512>;
            if (d <= 1536 && RDT != KDA_F32) run(DT, RDT, T128{}, std::integral_constant<int, 2>{});
            else if (d <= 2048) run(DT, RDT, T256{}, std::integral_constant<int, 1>{});
            else if (d <= 4096 && d > 3968 && R >= 16384 && RDT != KDA_F32) run(DT, RDT, T512{}, std::integral_constant<int, 1>{});
            else if (d <= 4096) run(DT, RDT, T256{}, std::integral_constant<int, 2>{});
            else if (d <= 8192) run(DT, RDT, T512{}, std::integral_constant<int, 2>{});
            else run(DT, RDT, T512{}, std::integral_constant<int, 4>{});
        };
        using BF = std::integral_constant<int, KDA_BF16>;
        using HF = std::integral_constant<int, KDA_F16>;
        using F = std::integral_constant<int, KDA_F32>;
        if (in_dtype == KDA_F32) by_len(F{}, F{});
        else if (in_dtype == KDA_BF16) residual_dtype == KDA_F32 ? by_len(BF{}, F{}) : by_len(BF{}, BF{});
        else residual_dtype == KDA_F32 ? by_len(HF{}, F{}) : by_len(HF{}, HF{});
        return err == cudaSuccess ? launch_status() : runtime_failed();
    }
    with_types(in_dtype, vec, [&](auto DT, auto V) {
        with_row_form<V>((d + 7) / 8, R < 1024, [&](auto TPR, auto NV) {
            constexpr int rows = norm_threads(TPR) / TPR;
            residual_norm_kernel<DT, V, TPR, NV><<<(unsigned)(((int64_t)R + rows - 1) / rows), norm_threads(TPR), 0, s>>>(a);
        });
    });
    return launch_status();
}
