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
// Bound by HBM: the state's bytes.  A warp holds whole rows of S^T in registers (a row = one value channel, 128 key
// channels), asked for at the start, so that the bytes in flight are the registers of all resident warps.
// 256 requests, 32 heads, fp32 states: one position 169 us (95 % of the measured copy rate); 64 requests of seven
// positions: verify 39 us (57 %), commit 54 us (76 %).
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

// e^g for what is not summed up over calls; a forgotten state leaves exactly nothing.
__device__ __forceinline__ float exp_of(float g) { return g <= -104.f ? 0.f : expf(g); }

// What a state is multiplied by.  The nearest fp32 value to e^g is up to 2^-25 off, for a fixed slope alike at every token:
// 9e-5 of the state after 4096 tokens at g = -1e-4.  So from e^g = 1/2 on it is taken less one, whose rounding goes by
// 1 - e^g, and an fp32 state s becomes s + s (e^g - 1), rounded once.  (16-bit states lose more at each store.)  256 requests,
// 32 heads: 159.7 us, with the product alone 158.9; 64 x 7 commit 49.6 and 48.7.
struct Fade {
    float m;    // e^g - 1 if near, else e^g
    bool near;
};
constexpr float kNear = -0.69f;
template <int ST>
__device__ __forceinline__ Fade fade_of(float g) { return ST == kStateF32 && g > kNear ? Fade{expm1f(g), true} : Fade{exp_of(g), false}; }
__device__ __forceinline__ float faded(float s, Fade f) {
    // an infinite s stays what it is: only a finite one is taken times e^g - 1
    return f.near ? fmaf(fminf(fmaxf(s, -3.402823466e38f), 3.402823466e38f), f.m, s) : s * f.m;
}
__device__ __forceinline__ float4 faded(float4 s, Fade f) {
    return make_float4(faded(s.x, f), faded(s.y, f), faded(s.z, f), faded(s.w, f));
}

// One position: 32 rows a block, eight a warp.  Nothing is shared between warps.  Seven blocks a SM by registers (64 of them):
// 16-bit states, 256 requests, 94.7 us, with the 72 that the compiler takes otherwise 99.5.
template <int ST>
__global__ void __launch_bounds__(kDecayThreads, 7) decay_step_kernel(const DecayDecodeArgs a) {
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
        const Fade fade = fade_of<ST>(log_decay_of(a.head_decay, a.log_decay, r, a.H, h));
        if (a.out.base) {
            float4 q = load4_as(row_of(a.q, r, hk, a.in_dt), 4 * lane, a.in_dt);
            q = make_float4(q.x * a.scale, q.y * a.scale, q.z * a.scale, q.w * a.scale);
            const float kq = warp_sum(f4_dot(k, q));
            float d[RW];
#pragma unroll
            for (int i = 0; i < RW; ++i) d[i] = f4_dot(s[i], q);
            const float o = fmaf(fade.near ? 1.f + fade.m : fade.m, reduce_scatter<RW>(d, lane), kq * vm);
            if ((lane & 3) == 0) store1_as(out_row(a.out, r, h, a.out_dt), row0 + (lane >> 2), o, a.out_dt);
        }
        if (p.commit) {
            if (fade.near) {
#pragma unroll
                for (int i = 0; i < RW; ++i) s[i] = f4_fma(__shfl_sync(0xffffffffu, vm, 4 * i), k, faded(s[i], fade));
            } else {
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    const float4 x = f4_mul(s[i], make_float4(fade.m, fade.m, fade.m, fade.m));
                    s[i] = f4_fma(__shfl_sync(0xffffffffu, vm, 4 * i), k, x);
                }
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

// D += A B of 16 x 8 x 8 in tf32 (fp32 bits whose lower 13 are not looked at), fp32 sums.  Lane 4 g + c has rows g and
// g + 8 of A and D; columns (of A: the k index) c and c + 4 of A, and c, c + 4 by n = g of B; columns 2c, 2c + 1 of D.
__device__ __forceinline__ void mma_tf32(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}
__device__ __forceinline__ float tf32_of(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }

// Sixteen rows times eight, over 4 + 4 of their 128 channels a step pair: x and y (rows g and g + 8) are the lane's
// channels 4c .. 4c + 3 of a group of 16, q those of row g of the other side, whose order the products may choose.
// The rows go in two parts of 11 bits each, 2^-21 of them left out; q is exact in one (bf16, fp16) or in two, too.
// N sums take the products in turns: on one sum 32 of them waited for one another, some 35 cycles each.
template <int N>
__device__ __forceinline__ void rows_times(float (&d)[N][4], float4 x, float4 y, float4 q, bool wide) {
    const float4 xh = make_float4(tf32_of(x.x), tf32_of(x.y), tf32_of(x.z), tf32_of(x.w));
    const float4 yh = make_float4(tf32_of(y.x), tf32_of(y.y), tf32_of(y.z), tf32_of(y.w));
    mma_tf32(d[0], xh.x, yh.x, xh.y, yh.y, q.x, q.y);
    mma_tf32(d[1 % N], xh.z, yh.z, xh.w, yh.w, q.z, q.w);
    mma_tf32(d[2 % N], x.x - xh.x, y.x - yh.x, x.y - xh.y, y.y - yh.y, q.x, q.y);
    mma_tf32(d[3 % N], x.z - xh.z, y.z - yh.z, x.w - xh.w, y.w - yh.w, q.z, q.w);
    if (wide) {
        mma_tf32(d[2 % N], xh.x, yh.x, xh.y, yh.y, q.x - tf32_of(q.x), q.y - tf32_of(q.y));
        mma_tf32(d[3 % N], xh.z, yh.z, xh.w, yh.w, q.z - tf32_of(q.z), q.w - tf32_of(q.w));
    }
}
template <int N>
__device__ __forceinline__ float sum_of(const float (&d)[N][4], int e) {
    return N == 4 ? (d[0][e] + d[1 % N][e]) + (d[2 % N][e] + d[3 % N][e]) : d[0][e] + d[1 % N][e];
}

// Several positions: a block or two a (request, head), sixteen value channels a warp.  Lane 4 g + c has rows g and g + 8 of
// its warp's, and of them channels 4c .. 4c + 3 of each group of 16 key channels: the operand layout of the warp's
// tensor-core products with the positions' queries, which take the place of a sum over the warp for each (row,
// position): with those, the verify of seven positions of 64 requests, 32 heads, took 104 us, most of it instructions;
// now 39, and what is left is a block's own chain (rows, then state, then products, then rows out) at two blocks a SM,
// which their registers allow.  The state itself is updated by fp32 FMAs, each rounded to nearest.  In shared
// memory: the positions' rows, their products q_t . k_j with the decays between.
template <int ST, int NT, int PARTS>  // NT: groups of eight positions; PARTS: blocks a (request, head)
__global__ void __launch_bounds__(256 / PARTS, 2 * PARTS) decay_steps_kernel(const DecayDecodeArgs a) {
    using SIO = State<ST>;
    constexpr int kWarps = 8 / PARTS, kRows = 16 * kWarps;  // of a block: warps, value channels
    constexpr int KT = 8 * NT, QS = 144, KS = 136;  // row lengths in shared memory that spread the lanes' reads over all banks
    __shared__ __align__(16) float sq[KT][QS], sk[KT][KS], sv[KT][kRows];
    __shared__ float w[KT][KT + 1], lead[KT], dec[KT], logs[KT], kept[KT], sum_log;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int unit = blockIdx.x / PARTS, part = blockIdx.x % PARTS;
    const int r = unit / a.H, h = unit - r * a.H, hk = h / a.group;
    const Plan p = plan_of(a, r, tid == 0 && part == 0 && h == 0);
    const int ql = p.ql, nc = p.commit, col = 16 * warp + g, row = part * kRows + col;
    const bool answer = a.out.base != nullptr, wide = a.in_dt == KDA_F32;
    const bool moved = p.live && p.dst >= 0 && p.dst != p.src;
    const int64_t first = (int64_t)r * a.K;
    // the positions' rows are asked for ahead of the state, whose 64 KiB they would else queue behind: what is made of
    // them alone is then done while the state comes
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kTurns = KT / kWarps;  // rows t of a warp: warp, warp + kWarps, ..
    float4 qr[kTurns], kr[kTurns], vr[kTurns];
    float log_a = 0.f;
    if (ql) {
        if (tid < ql) log_a = log_decay_of(a.head_decay, a.log_decay, first + tid, a.H, h);
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int t = warp + kWarps * i;
            const bool there = t < ql;
            kr[i] = there ? load4_as(row_of(a.k, first + t, hk, a.in_dt), 4 * lane, a.in_dt) : zero;
            vr[i] = there && 4 * lane < kRows ? load4_as(row_of(a.v, first + t, h, a.in_dt), part * kRows + 4 * lane, a.in_dt) : zero;
            qr[i] = there && answer ? load4_as(row_of(a.q, first + t, hk, a.in_dt), 4 * lane, a.in_dt) : zero;
        }
    }
    float4 s[2][8];
    if ((ql && answer) || nc || moved) {
        const size_t S = state_elem(p.src, a.H, h) + (size_t)row * kD + 4 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 8; ++x) s[i][x] = SIO::load4_cs(a.pool, S + (size_t)(8 * i) * kD + 16 * x);
    }
    for (int t = ql + warp; answer && t < a.K; t += kWarps)  // positions that there are not
        for (int i = lane; i < kRows; i += 32) store1_as(out_row(a.out, first + t, h, a.out_dt), part * kRows + i, 0.f, a.out_dt);
    if (ql) {
        if (tid < ql) dec[tid] = exp_of(log_a), logs[tid] = log_a;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int t = warp + kWarps * i;
            *reinterpret_cast<float4*>(&sk[t][4 * lane]) = kr[i];
            if (4 * lane < kRows) *reinterpret_cast<float4*>(&sv[t][4 * lane]) = vr[i];
            *reinterpret_cast<float4*>(&sq[t][4 * lane]) = qr[i];
        }
        __syncthreads();
        // thread j: prod_{j<s<=t} a_s for t >= j; the decays from the state; 0 for t < j
        if (tid < KT) {
            const int j = tid;
            float de[KT];
#pragma unroll
            for (int t = 0; t < KT; ++t) de[t] = t < ql ? dec[t] : 0.f;
            float f = j < ql ? 1.f : 0.f, l = 1.f;
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                if (t > j) f *= de[t];
                if (t <= j) l *= de[t];
                w[t][j] = t < j ? 0.f : f;
            }
            lead[j] = l;
            kept[j] = nc ? w[nc - 1][j] : 0.f;  // of v_j in the committed state
            if (j == nc - 1) {
                float g = 0.f;
                for (int t = 0; t < nc; ++t) g += logs[t];
                sum_log = g;
            }
        }
        // keys 0 .. 15 times eight queries a warp, of the last warps, while the state is on its way
        constexpr int kSums = NT == 1 ? 4 : 2;
        const int kn = warp - (kWarps - NT);
        float kq[kSums][4];
        if (answer && kn >= 0) {
#pragma unroll
            for (int i = 0; i < kSums; ++i) kq[i][0] = kq[i][1] = kq[i][2] = kq[i][3] = 0.f;
#pragma unroll 2
            for (int x = 0; x < 8; ++x) {
                const int at = 16 * x + 4 * c;
                rows_times<kSums>(kq, *reinterpret_cast<const float4*>(&sk[g][at]), NT == 1 ? zero : *reinterpret_cast<const float4*>(&sk[(g + 8) % KT][at]),
                                  *reinterpret_cast<const float4*>(&sq[8 * kn + g][at]), wide);
            }
        }
        __syncthreads();
        float d[NT][kSums][4];
        if (answer) {
            if (kn >= 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = g + 8 * (e >> 1), t = 8 * kn + 2 * c + (e & 1);
                    if (j < KT) w[t][j] *= sum_of<kSums>(kq, e);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4 * kSums; ++e) d[n][e >> 2][e & 3] = 0.f;
#pragma unroll
            for (int x = 0; x < 8; ++x)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    rows_times<kSums>(d[n], s[0][x], s[1][x], *reinterpret_cast<const float4*>(&sq[8 * n + g][16 * x + 4 * c]), wide);
        }
        if (answer) {
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int t = 8 * n + 2 * c;
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = lead[t + (e & 1)] * sum_of<kSums>(d[n], e);
                for (int j = 0; j < ql; ++j) {
                    const float w0 = w[t][j], w1 = w[t + 1][j], v0 = sv[j][col], v1 = sv[j][col + 8];
                    if (j <= t) o[0] = fmaf(w0, v0, o[0]), o[2] = fmaf(w0, v1, o[2]);
                    if (j <= t + 1) o[1] = fmaf(w1, v0, o[1]), o[3] = fmaf(w1, v1, o[3]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t + (e & 1) < ql)
                        store1_as(out_row(a.out, first + t + (e & 1), h, a.out_dt), row + 8 * (e >> 1), a.scale * o[e], a.out_dt);
            }
        }
        if (nc) {
            // (far from one, the product of the positions' decays: it is as exact, and needs no sum)
            const float g = sum_log;
            const Fade f = ST == kStateF32 && g > kNear ? Fade{expm1f(g), true} : Fade{lead[nc - 1], false};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < 8; ++x) s[i][x] = faded(s[i][x], f);
            for (int j = 0; j < nc; ++j) {
                const float v0 = kept[j] * sv[j][col], v1 = kept[j] * sv[j][col + 8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float4 k = *reinterpret_cast<const float4*>(&sk[j][16 * x + 4 * c]);
                    s[0][x] = f4_fma(v0, k, s[0][x]);
                    s[1][x] = f4_fma(v1, k, s[1][x]);
                }
            }
        }
    }
    if (p.live && p.dst >= 0 && (nc || moved)) {
        const size_t S = state_elem(p.dst, a.H, h) + (size_t)row * kD + 4 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 8; ++x) SIO::store4_cs(a.pool, S + (size_t)(8 * i) * kD + 16 * x, s[i][x]);
    }
}

template <int ST>
void launch(const DecayDecodeArgs& a, cudaStream_t s) {
    const unsigned units = (unsigned)a.R * (unsigned)a.H;
    if (a.K == 1)
        decay_step_kernel<ST><<<units * 4, kDecayThreads, 0, s>>>(a);
    // A state in two blocks of 64 value channels: four chains a SM for two, and the positions' rows read twice.  64 requests
    // of 32 heads, fp32 states, two blocks and one: step of 2 positions 56 and 62 us, 4 58 and 63; verify 4 35.2 and 36.9,
    // 5 41.3 and 36.9, 7 40.4 and 36.6; commit 4 45 and 48.5, 7 50.5 and 51.5.  bf16 states, 7: commit 38.5 and 37.1.
    // Steps of 5 to 8 positions go with the verify, which the host does not tell from them: of 7, 66.5 and 66.8 (256
    // requests 273.7 and 275), bf16 states 58.2 and 56.4 (246 and 231), but fp32 rows 63.9 and 68.1 (227 and 249).
    else if (a.K <= 4 || (a.K <= 8 && !a.out.base && ST == kStateF32))
        decay_steps_kernel<ST, 1, 2><<<units * 2, 128, 0, s>>>(a);
    else if (a.K <= 8)
        decay_steps_kernel<ST, 1, 1><<<units, 256, 0, s>>>(a);
    else
        decay_steps_kernel<ST, 2, 1><<<units, 256, 0, s>>>(a);
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
    KDA_REQUIRE(decays_ok(head_decay, log_decay), KDA_ERR_INVALID_ARG);
    const void* need[] = {state_pool, slot};
    for (const void* p : need) KDA_REQUIRE(p != nullptr, KDA_ERR_INVALID_ARG);
    const void* ptrs[] = {state_pool, slot, dst_slot, q_len, n_commit};
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
