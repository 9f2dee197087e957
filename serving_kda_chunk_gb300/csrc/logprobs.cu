// logprobs.cu -- kda_token_logprobs: log probability of given tokens, entropy and top
// alternatives of logits rows.
//
// One pass over the logits, which is what bounds it (HBM).  A thread keeps, over its elements and
// relative to a reference v of its own (moved when an element exceeds it by 8 ln2),
//   z = sum 2^d,  w = sum 2^d d,  d = (x - v) log2 e
// and its largest element; the block joins them to
//   logprob = (x_token - max) - ln z,  entropy = ln2 (log2 z - w / z)    (relative to the maximum).
//
// Top ids without a second pass: elements lie in columns, column t being thread t's.  A threshold
// that at least k column maxima reach is reached by the top k elements as well, and only by elements
// of those columns.  Each column also leaves the maximum of every piece of it (8 vectors, more in the
// longest rows) in shared memory, so only the pieces that reach the threshold are read again: about k
// times 128 bytes.  (Reading the columns again whole cost a quarter of the time: strided, and by then
// out of L2.)  The few elements at or above the threshold are ranked by (value, -id).
// Ties at the threshold can make them many (a mask of -inf over most of a vocabulary): then
// the columns' maxima take part with their ids, and the k best elements are drawn one after another,
// the column that gave one being read again for its next.
//
// Few rows: a row is split over a cluster of up to 8 blocks, whose sums and lists the first joins
// through distributed shared memory.
#include <cooperative_groups.h>

#include "kda_host.h"
#include "latent_common.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

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

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kCand = 256;      // candidates of the ranked path
constexpr int kPieces = 128;    // pieces of columns it reads again
constexpr int kBatch = 8;       // vectors of a column asked for at once
constexpr int kMaxSeg = 32;     // pieces of a column
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kFloor = -200.f;  // 2^-200 is 0 in fp32: below this an element adds nothing

// A value as an unsigned number of the same order; -0 equals +0 and NaN lies below -inf.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return x != x ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
// (value, id) as one key: larger value first, then smaller id; 0 is below every element's
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t id) { return ((uint64_t)order << 32) | (uint32_t)~id; }

// 16 bytes of a row: unpacking, and their largest element (NaN if one is NaN)
template <int DT>
struct Vec {
    static constexpr int n = 8;
    static __device__ __forceinline__ void unpack(uint4 v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = Elem<DT>::get2(w[i]);
            x[2 * i] = p.x;
            x[2 * i + 1] = p.y;
        }
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        if constexpr (DT == KDA_BF16)
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else
            asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float max_of(uint4 v) {
        const float2 p = Elem<DT>::get2(max2(max2(v.x, v.y), max2(v.z, v.w)));
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(p.x), "f"(p.y));
        return r;
    }
};
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
template <>
struct Vec<KDA_F32> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void unpack(uint4 v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float max_of(uint4 v) {
        return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                       max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
};

// The running sums of a thread.  The difference is taken before the factor: products of values near
// the type's largest would overflow, and near the maximum the difference is exact.
struct Sums {
    float v = 0.f;                                  // reference
    float limit = -__builtin_huge_valf();           // an element above this moves it
    float2 z = {0.f, 0.f}, w = {0.f, 0.f};
    __device__ __forceinline__ void raise(float vmax) {
        if (z.x + z.y > 0.f) {  // else nothing yet, whatever v was
            const float d = fmaxf((v - vmax) * kLog2e, kFloor), f = ex2(d);
            w = make_float2(f * (w.x + z.x * d), f * (w.y + z.y * d));
            z = make_float2(f * z.x, f * z.y);
        }
        v = vmax;
        limit = vmax + 8.f * kLn2;
    }
    __device__ __forceinline__ void add2(float a, float b) {
        float2 d = __fadd2_rn(make_float2(a, b), make_float2(-v, -v));
        d = __fmul2_rn(d, make_float2(kLog2e, kLog2e));
        d.x = fmaxf(d.x, kFloor);
        d.y = fmaxf(d.y, kFloor);
        const float2 e = make_float2(ex2(d.x), ex2(d.y));
        z = __fadd2_rn(z, e);
        w = __ffma2_rn(e, d, w);
    }
};

struct LpShared {
    float m[kLpWarps], z[kLpWarps], w[kLpWarps];
    float bm, bz, bw;                  // the block's: maximum (NaN possible), sums relative to it
    alignas(16) uint32_t col[kLpThreads];          // column maxima as ordered numbers
    uint64_t ckey[kLpWarps];
    uint32_t tau;
    int n_pieces, n_cand;
    int pieces[kPieces];               // piece * kLpThreads + column
    uint64_t cand[kCand];
    uint64_t list[kMaxTop];            // the block's top keys, descending
};

template <int DT>
__global__ void __launch_bounds__(kLpThreads) logprob_kernel(const __grid_constant__ LogprobArgs a, const int C, const int per) {
    using E = Elem<DT>;
    using T = typename E::T;
    using X = Vec<DT>;
    constexpr int VE = X::n;
    __shared__ LpShared s;
    extern __shared__ float seg[];  // [pieces][kLpThreads] maxima
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float inf = __int_as_float(0x7f800000);
    const int64_t r = blockIdx.x / C;
    const int part = blockIdx.x % C;
    const T* row = static_cast<const T*>(a.logits) + r * a.row_stride;
    // head elements up to a 16-byte boundary, vectors, tail elements; the vectors are cut over the
    // blocks, the head goes to the first and the tail to the last
    const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int head = min(a.V, mis ? VE - mis : 0);
    const int nv = (a.V - head) / VE;
    const int v0 = (int)((int64_t)nv * part / C), v1 = (int)((int64_t)nv * (part + 1) / C);
    const int n_head = part == 0 ? head : 0;
    const int tail0 = head + nv * VE, n_tail = part == C - 1 ? a.V - tail0 : 0;
    const uint4* vec = reinterpret_cast<const uint4*>(row + head);

    // the token's logit, asked for ahead of the pass
    const int tok = tid == 0 && part == 0 ? a.tokens[r] : -1;
    const float x_tok = tok >= 0 && tok < a.V ? E::get(row[tok]) : 0.f;
    Sums su;
    float cm = -inf;  // this column's maximum, NaN if it holds one
    auto one = [&](int i) {
        const float x = E::get(row[i]);
        cm = max_nan(cm, x);
        if (x > su.limit) su.raise(x);
        su.add2(x, -inf);
    };
    auto take = [&](uint4 v) {
        const float vm = X::max_of(v);
        if (vm > su.limit) su.raise(vm);
        float x[VE];
        X::unpack(v, x);
#pragma unroll
        for (int i = 0; i < VE; i += 2) su.add2(x[i], x[i + 1]);
        return vm;
    };
    if (tid < n_head) one(tid);
    if (tid < n_tail) one(tail0 + tid);
    float pm = cm;  // the piece's maximum; the head and tail elements belong to piece 0
    cm = -inf;
    const int batches = (v1 - v0 + kBatch * kLpThreads - 1) / (kBatch * kLpThreads);
    for (int b = 0, in = 0, sg = 0; b < batches; ++b) {
        const int j = v0 + b * (kBatch * kLpThreads) + tid;
        float bm = -inf;
        if (j + (kBatch - 1) * kLpThreads < v1) {
            uint4 v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) v[u] = __ldcs(vec + j + u * kLpThreads);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) bm = max_nan(bm, take(v[u]));
        } else {
            for (int q = j; q < v1; q += kLpThreads) bm = max_nan(bm, take(__ldg(vec + q)));
        }
        pm = max_nan(pm, bm);
        if (++in == per || b + 1 == batches) {
            seg[sg * kLpThreads + tid] = pm;
            cm = max_nan(cm, pm);
            pm = -inf;
            in = 0;
            ++sg;
        }
    }
    cm = max_nan(cm, pm);  // a row without a whole vector
    const int n_seg = (batches + per - 1) / per;

    // ---- the block's sums, relative to its maximum
    const uint32_t mine = order_of(cm);
    float bmax;
    {
        bmax = cm;
#pragma unroll
        for (int o = 16; o; o >>= 1) bmax = max_nan(bmax, __shfl_xor_sync(~0u, bmax, o));
        if (lane == 0) s.m[warp] = bmax;
        s.col[tid] = mine;
        if (tid == 0) {
            s.n_pieces = s.n_cand = 0;
        }
        __syncthreads();
        bmax = s.m[0];
#pragma unroll
        for (int i = 1; i < kLpWarps; ++i) bmax = max_nan(bmax, s.m[i]);
        const float d = fmaxf((su.v - bmax) * kLog2e, kFloor), tz = su.z.x + su.z.y;
        const float f = ex2(d);
        float z = tz > 0.f ? f * tz : 0.f, w = tz > 0.f ? f * ((su.w.x + su.w.y) + tz * d) : 0.f;
        warp_sum2(z, w);
        if (lane == 0) {
            s.z[warp] = z;
            s.w[warp] = w;
        }
        __syncthreads();
        if (tid == 0) {
            z = w = 0.f;
#pragma unroll
            for (int i = 0; i < kLpWarps; ++i) z += s.z[i], w += s.w[i];
            s.bm = bmax;
            s.bz = z;
            s.bw = w;
        }
    }

    // ---- the block's top keys
    const int top = a.top;
    // every element of column c, split over a warp's lanes: f(value, id)
    auto column = [&](int c, auto f) {
        if (lane == 0 && c < n_head) f(E::get(row[c]), c);
        if (lane == 0 && c < n_tail) f(E::get(row[tail0 + c]), tail0 + c);
        for (int q = v0 + c + lane * kLpThreads; q < v1; q += 32 * kLpThreads) {
            float x[VE];
            X::unpack(__ldg(vec + q), x);
#pragma unroll
            for (int i = 0; i < VE; ++i) f(x[i], head + q * VE + i);
        }
    };
    if (top > 0) {
        if (warp == 0) {
            // a threshold that at least `top` column maxima reach and not many more: bit by bit from
            // the highest in which they differ (the bits above are common to all)
            uint32_t o[kLpThreads / 32], any = 0, all = ~0u;
#pragma unroll
            for (int i = 0; i < kLpThreads / 32; ++i) {
                o[i] = s.col[i * 32 + lane];
                any |= o[i];
                all &= o[i];
            }
            any = __reduce_or_sync(~0u, any);
            all = __reduce_and_sync(~0u, all);
            const uint32_t differ = any ^ all;
            uint32_t t = differ ? all & ~(0xffffffffu >> __clz(differ)) : all;
            for (uint32_t bit = differ ? 0x80000000u >> __clz(differ) : 0; bit; bit >>= 1) {
                int n = 0;
#pragma unroll
                for (int i = 0; i < kLpThreads / 32; ++i) n += o[i] >= (t | bit);
                n = __reduce_add_sync(~0u, n);
                if (n >= top) {
                    t |= bit;
                    if (n <= top + top / 2) break;
                }
            }
            if (lane == 0) s.tau = t;
        }
        __syncthreads();
        const uint32_t tau = s.tau;
        const float floor = value_of(tau);
        if (mine >= tau) {
            for (int g = 0; g < max(n_seg, 1); ++g) {
                if (n_seg > 0 && !(seg[g * kLpThreads + tid] >= floor)) continue;
                const int at = atomicAdd(&s.n_pieces, 1);
                if (at < kPieces) s.pieces[at] = g * kLpThreads + tid;
            }
        }
        if (tid < kMaxTop) s.list[tid] = 0;
        __syncthreads();
        const int n_pieces = bmax != bmax ? kPieces + 1 : s.n_pieces;  // a column with NaN has no rank
        if (n_pieces <= kPieces) {
            auto keep = [&](float x, int id) {
                const uint32_t o = order_of(x);
                if (o >= tau) {
                    const int at = atomicAdd(&s.n_cand, 1);
                    if (at < kCand) s.cand[at] = key_of(o, (uint32_t)id);
                }
            };
            // eight lanes a piece
            for (int i = tid >> 3; i < n_pieces; i += kLpThreads / 8) {
                const int g = s.pieces[i] / kLpThreads, c = s.pieces[i] % kLpThreads;
                if (g == 0 && (tid & 7) == 0) {
                    if (c < n_head) keep(E::get(row[c]), c);
                    if (c < n_tail) keep(E::get(row[tail0 + c]), tail0 + c);
                }
                const int end = min(v1, v0 + (g + 1) * per * kBatch * kLpThreads);
                for (int q = v0 + (g * per * kBatch + (tid & 7)) * kLpThreads + c; q < end; q += 8 * kLpThreads) {
                    const uint4 v = __ldg(vec + q);
                    if (X::max_of(v) < floor) continue;
                    float x[VE];
                    X::unpack(v, x);
#pragma unroll
                    for (int e = 0; e < VE; ++e) keep(x[e], head + q * VE + e);
                }
            }
        }
        __syncthreads();
        const int n = s.n_cand;
        if (n_pieces <= kPieces && n <= kCand) {
            // keys are distinct, so every rank is taken once
            if (tid < n) {
                const uint64_t k = s.cand[tid];
                int rk = 0;
                for (int i = 0; i < n; ++i) rk += s.cand[i] > k;
                if (rk < top) s.list[rk] = k;
            }
        } else {
            // one after another: `best` is this column's largest key below the last one drawn
            uint64_t best = 0;
            auto better = [&](float x, int id, uint64_t below, uint64_t& b) {
                const uint64_t k = key_of(order_of(x), (uint32_t)id);
                if (k < below && k > b) b = k;
            };
            if (tid < n_head) better(E::get(row[tid]), tid, ~0ull, best);
            if (tid < n_tail) better(E::get(row[tail0 + tid]), tail0 + tid, ~0ull, best);
            for (int q = v0 + tid; q < v1; q += kLpThreads) {
                float x[VE];
                X::unpack(__ldg(vec + q), x);
#pragma unroll
                for (int i = 0; i < VE; ++i) better(x[i], head + q * VE + i, ~0ull, best);
            }
            for (int k = 0; k < top; ++k) {
                uint64_t b = best;
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    const uint64_t y = __shfl_xor_sync(~0u, b, o);
                    b = y > b ? y : b;
                }
                if (lane == 0) s.ckey[warp] = b;
                __syncthreads();
                uint64_t win = s.ckey[0];
#pragma unroll
                for (int i = 1; i < kLpWarps; ++i) win = s.ckey[i] > win ? s.ckey[i] : win;
                if (win == 0) break;  // fewer elements than places
                if (tid == 0) s.list[k] = win;
                const uint32_t who = __ballot_sync(~0u, best == win);
                if (who) {  // the warp of the column that gave it
                    const int c = warp * 32 + __ffs(who) - 1;
                    uint64_t nb = 0;
                    column(c, [&](float x, int id) { better(x, id, win, nb); });
#pragma unroll
                    for (int o = 16; o; o >>= 1) {
                        const uint64_t y = __shfl_xor_sync(~0u, nb, o);
                        nb = y > nb ? y : nb;
                    }
                    if (tid == c) best = nb;
                }
                __syncthreads();
            }
        }
    }

    // ---- the row's results: the first block joins the cluster's
    float m, z, w;
    uint64_t key = 0;
    int rank = tid;
    cg::cluster_group cluster = cg::this_cluster();
    if (C > 1) {
        cluster.sync();
        if (part == 0) {
            m = s.bm;
            for (int c = 1; c < C; ++c) m = max_nan(m, cluster.map_shared_rank(&s, c)->bm);
            z = w = 0.f;
            for (int c = 0; c < C; ++c) {
                const LpShared* o = cluster.map_shared_rank(&s, c);
                const float d = fmaxf((o->bm - m) * kLog2e, kFloor), oz = o->bz;
                const float f = ex2(d);
                z += oz > 0.f ? f * oz : 0.f;
                w += oz > 0.f ? f * (o->bw + oz * d) : 0.f;
            }
            if (top > 0) {
                __syncthreads();
                if (tid < C * kMaxTop) key = cluster.map_shared_rank(&s, tid / kMaxTop)->list[tid % kMaxTop];
                static_assert(8 * kMaxTop <= kCand && 8 * kMaxTop <= kLpThreads, "a thread a key");
                s.cand[tid] = key;
                __syncthreads();
                rank = 0;
                for (int i = 0; i < C * kMaxTop; ++i) rank += s.cand[i] > key;
                if (key == 0) rank = kMaxTop;
            }
        }
        cluster.sync();  // the others' shared memory has been read
        if (part != 0) return;
    } else {
        __syncthreads();
        m = s.bm;
        z = s.bz;
        w = s.bw;
        if (tid < kMaxTop) key = s.list[tid];
    }
    const float nan = __int_as_float(0x7fffffff);
    const bool none = !(z > 0.f) || !(m < inf);  // only -inf, or +inf or NaN in the row
    const float lz = none ? nan : log2f(z);
    if (tid == 0) {
        float lp = 0.f;
        if (tok >= a.V) report(a.dev_status, KDA_DEV_BAD_SLOT);
        else if (tok >= 0) lp = (x_tok - m) - lz * kLn2;
        a.logprob[r] = lp;
        if (a.entropy) a.entropy[r] = (lz - w / z) * kLn2;
    }
    if (rank < top && key != 0) {
        const int id = (int)~(uint32_t)key;
        a.top_ids[r * top + rank] = id;
        a.top_logprobs[r * top + rank] = (value_of((uint32_t)(key >> 32)) - m) - lz * kLn2;
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
    KDA_REQUIRE(top <= kMaxTop && top <= V && R < (1 << 28), KDA_ERR_UNSUPPORTED);
    if (R == 0) return KDA_OK;
    KDA_REQUIRE(logits != nullptr && reinterpret_cast<uintptr_t>(logits) % dtype_bytes(dtype) == 0,
                KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(row_stride >= V || (R == 1 && row_stride >= 0), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(tokens != nullptr && logprob != nullptr, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(top == 0 || (top_ids != nullptr && top_logprobs != nullptr), KDA_ERR_INVALID_ARG);
    const void* ptrs[] = {tokens, logprob, entropy, top_ids, top_logprobs, dev_status};
    for (const void* p : ptrs) KDA_REQUIRE(aligned16(p), KDA_ERR_INVALID_ARG);
    const LogprobArgs a{logits, row_stride, V, tokens, logprob, entropy, top, top_ids, top_logprobs, dev_status};
    // blocks a row: enough rows fill the SMs by themselves (splitting 448 rows in two: 33 -> 45 us);
    // else split, down to 16 vectors a thread (one row of 32768: 7.7 us in one block, 8.3 in two, 10.3 in
    // eight; 32 rows of 160000: 12.3 us in four, 14.4 in eight or two)
    int C = 1;
    while (C < 8 && (int64_t)R * C < 304 && (int64_t)V * dtype_bytes(dtype) >= 2ll * C * kLpThreads * 256) C *= 2;
    // batches of a block's share, at most kMaxSeg pieces of them
    const int64_t batches = ((int64_t)V * dtype_bytes(dtype) / 16 / C + 1 + kBatch * kLpThreads - 1) / (kBatch * kLpThreads);
    const int per = (int)((batches + kMaxSeg - 1) / kMaxSeg);
    const int pieces = (int)((batches + per - 1) / per);
    auto* f = dtype == KDA_BF16 ? logprob_kernel<KDA_BF16> : dtype == KDA_F16 ? logprob_kernel<KDA_F16> : logprob_kernel<KDA_F32>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(R * C));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = (size_t)pieces * kLpThreads * sizeof(float);
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = C > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, f, a, C, per) != cudaSuccess) return runtime_failed();
    return launch_status();
}
