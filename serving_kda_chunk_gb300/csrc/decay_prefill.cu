// decay_prefill.cu -- kda_decay_prefill: linear attention with a decay a head over packed sequences.
//
// Chunks of 128 tokens.  With G_i the sum of the log decays up to token i of the chunk (S_0 the state before it):
//     o_i = scale ( sum_{j<=i} e^{G_i - G_j} (q_i . k_j) v_j + e^{G_i} S_0^T q_i ),
//     S_C = e^{G_C} S_0 + sum_j e^{G_C - G_j} k_j v_j^T.
// Four products of 128 x 128 x 128 a chunk and head on the tensor cores (tcgen05, accumulators in tensor memory):
//     scores Q K^T;  Q S_0;  P V with the weighted, masked scores P, onto the last;  K~ V with the decayed keys K~.
// The last does not depend on the state, so the chain from chunk to chunk is S <- a S + K~ V in registers (a thread
// has a key channel and 64 value channels), and the state never collects the products' own rounding.
//
// What is rounded to the input type, and why that is enough: P and S_0, once each, for a product that is then
// rounded to a 16-bit output (their errors lie on the two summands of o, so together they weigh as much as the
// output's own rounding).  The decayed keys enter the fp32 state: they are split into parts of the input type, three
// for bf16 (by truncation, nothing left), two for fp16 (2^-22 left), and K~ V is as many products: part 1 and 2 as
// operand from tensor memory, part 3 from shared memory.  fp16 scores and states are scaled by a power of two (a
// row's, a chunk's) to the upper end of fp16's range first.
//
// Decays are kept per block of 32 tokens: D_i = G_i - G_end(block) >= 0 and the blocks' totals, from a sum in
// 64 bits.  A weight of an earlier block is then e^{G_i - G_end} (a row's factor) times e^{G_end - G_j} (a
// column's), both at most 1, and only the diagonal blocks take an exponential an element.  A forgotten state
// (-104 a token) inside a chunk leaves the differences exact enough: |D| is 150 a forgetting, in log2 units.
//
// Bound by HBM on paper: 128 KiB a chunk and head, 5700 cycles of an SM's share.  One CTA a SM, 16 warps: one loads
// (TMA; the next chunk into L2), one issues products, two sum decays in turns, four weigh scores and write results,
// eight split keys and carry the state.  Of shared memory K and V have two stages, Q and the state's operand one, the
// third part of K~ one (32 KiB each, 227 KB in all, so no second CTA); whole chunks of the input's type go out by TMA
// through the stage of their keys.  What bounds it now is instruction issue and fetch: the roles run different code on
// four schedulers, so what is rare is kept out of line, loops over halves stay loops, waits suspend their warp.  Each
// of the steps that made the code smaller gave more than one that took arithmetic away.  8 sequences of ~5182 tokens,
// 32 heads, bf16, states read and written: 281 to 290 us by the GPU, 4.9 to 5.1 of 6.7 TB/s (535 us in the first form that
// used tensor cores).
//
// Balance: the (sequence, head) pairs' chunks lie in one row, with places for what a pair costs besides, cut into equal
// ranges, one a CTA.  A pair cut once: the CTA that has its beginning takes that first and leaves the state for the next CTA, which takes its end
// last.  A pair over more CTAs: each but the last first sums up its range's own state (K and V only, read twice) and
// leaves it, then starts from the states before its own joined in order (131072 tokens, 16 heads: 612 to 639 us;
// with the pair's beginning in one pass the others waited for its state, 685 where this took 614; ranges weighted by their passes were slower
// too).  CTAs wait for one another, so this is a cooperative launch; every wait has a limit.
#include "decay_common.cuh"
#include "kda_host.h"
#include "latent_host.h"
#include "umma.cuh"

#include <algorithm>
#include <initializer_list>

namespace kda {
namespace {

using namespace umma;

constexpr int kDecayChunk = 128;
constexpr int kDecayCtas = 160;        // most CTAs of a cut launch (states that a workspace holds)
constexpr int kCutChunks = 6;          // a CTA's least range, in places: with 5, 6, 8, 10 one prompt of 16384 tokens, one head took 85, 81, 82,
                                       // 85 us, 6000 tokens of 16 heads 68, 66, 71, 78, two of 8192, 4 heads 70, 68, 72, 80.  5 is better
                                       // where 6 leaves SMs idle: 1500 tokens of 8 heads 45.2 and 50.5, 2500 of 4 47.2 and 50.4, four of
                                       // 2000, 2 heads 47.5 and 50.7, two of 2048, 8 heads 47.8 and 51.4, 4096 of 8 53.6 and 55.4
constexpr int kPreDecayThreads = 512;
constexpr int kShortUnit = 14;         // pairs of fewer places on average are not worth cutting while SMs are left: 1000 tokens of 16 heads
                                       // took 50 us cut, 39 not, 800 of 64 heads 46 and 41; 1500 of 8 heads (14 places) 52 and 53.  (A call
                                       // without a workspace, so without sums over lengths and a cooperative launch, takes 33, 34 and 43.)
constexpr int kUnitChunks = 2;         // what a pair's states, join and first chunk cost beside its chunks, for equal ranges: with 0, 1, 2,
                                       // 3 one prompt of 4096 tokens, 32 heads took 80, 76, 70, 72 us, 16 of 700, 16 heads 83, 73, 73, 74
constexpr uint32_t kTile = 32768;      // 128 rows of 128 16-bit channels
constexpr uint32_t kWaitLimit = 1u << 18;
constexpr uint32_t kFlagLimit = 1u << 21;

struct DecayPrefillArgs {
    LatentRows out;
    const float *head_decay, *log_decay;
    const int32_t *cu, *init_slot, *final_slot, *track_idx;
    void *pool, *track;
    int32_t* dev_status;
    int64_t P;
    int32_t N, T, H, group, M, hq, hk, hv, ho, out_dt, st;  // hq ..: 1, or 0 where all heads share a row
    bool boxes;  // output of the input's type: whole chunks are stored through maps.out
    float scale;
    int32_t give_up_cta, give_up_load;  // of the self-test: this CTA's loads stop before this chunk
    // of a cut launch: a flag and a decay a CTA, then the state it leaves
    uint32_t* flags;
    float* decays;
    float* states;
};

struct DecayMaps {
    CUtensorMap q, k, v, out;
};

// shared memory
constexpr uint32_t DS_K = 0, DS_V = 2 * kTile, DS_Q = 4 * kTile, DS_S = 5 * kTile, DS_LO = 6 * kTile, DS_G = 7 * kTile,
                   DS_TOT = DS_G + 2048, DS_BAR = DS_TOT + 160, DS_CTRL = DS_BAR + 8 * 28, DS_SCAN = DS_CTRL + 64,
                   DS_MAX = DS_SCAN + 136, DS_SCALE = DS_MAX + 64, DS_SMEM = DS_SCALE + 8;
static_assert(DS_SMEM <= 232448 && DS_SCAN % 8 == 0 && DS_BAR % 8 == 0, "shared memory plan");
constexpr int B_KF = 0, B_VF = 2, B_QF = 4, B_QK = 5, B_P = 6, B_SPLIT = 7, B_KV = 9, B_S = 11, B_QS = 12, B_SCALED = 13,
              B_O = 14, B_OFREE = 15, B_GF = 16, B_GFREE = 18, B_MEET = 20, B_FREE = 21, B_DRAIN = 23,
              B_NEVER = 24, B_TAKEN = 25, B_COUNT = 27;
// tensor memory: scores (their weights in the first half), results, K~ V, K~'s first two parts
constexpr uint32_t DT_SC = 0, DT_O = 128, DT_KV = 256, DT_K1 = 384, DT_K2 = 448;

// Chunks of a sequence, one for an empty one (its state is passed on), 0 for a refused one.
__device__ __forceinline__ int seq_chunks(const DecayPrefillArgs& a, int n, int& bad) {
    const int first = a.cu[n], last = a.cu[n + 1];
    bad = 0;
    if (first < 0 || last < first || last > a.T) bad |= KDA_DEV_BAD_SEQLEN;
    if ((a.init_slot && a.init_slot[n] >= a.P) || (a.final_slot && a.final_slot[n] >= a.P)) bad |= KDA_DEV_BAD_SLOT;
    return bad ? 0 : last == first ? 1 : (last - first + kDecayChunk - 1) / kDecayChunk;
}

enum PieceStart { kFromInit, kFromOthers, kFromZero };
enum PieceEnd { kNothing, kFinal, kPublish };

// Consecutive chunks c0 .. c1 - 1 of one (sequence, head).
struct Piece {
    int n, h, c0, c1, row0, rows;  // the sequence's first row and its rows
    bool state_only;
    int start, end;
};

// A CTA's range of chunks: from chunk fo of the first unit (a sequence and head) up to, but without, chunk lx of the last.
struct Range {
    int fn, fh, fo, ln, lh, lx;
    bool twice;  // the last unit goes on beyond the next CTA
};

// The pieces of a range in the order they are taken (see the top).
struct Pieces {
    Range r;
    int phase = 0, n, h;
    __device__ explicit Pieces(const Range& x) : r(x), n(x.fn), h(x.fh) {}
    __device__ __forceinline__ bool emit(const DecayPrefillArgs& a, Piece& p, int n_, int h_, int c0, int c1, bool only,
                                         int start, int end) {
        p.n = n_, p.h = h_, p.c0 = c0, p.c1 = c1, p.state_only = only, p.start = start, p.end = end;
        p.row0 = a.cu[n_];
        p.rows = a.cu[n_ + 1] - p.row0;
        return true;
    }
    __device__ __forceinline__ void step(const DecayPrefillArgs& a) {
        int bad;
        if (++h < a.H) return;
        h = 0;
        do ++n;
        while (n < a.N && n <= r.ln && seq_chunks(a, n, bad) == 0);
    }
    // (not inlined: its copies were a fourth of the kernel)
    __device__ __noinline__ bool next(const DecayPrefillArgs& a, Piece& p) {
        int bad;
        const bool same = r.fn == r.ln && r.fh == r.lh;
        // what goes on beyond this range and the next is gone through twice, for its state first (1 and 2; 3: a range within
        // a unit)
        if (phase == 0) {
            if (same && r.fo > 0) {
                phase = 3;
                return emit(a, p, r.fn, r.fh, r.fo, r.lx, true, kFromZero, kPublish);
            }
            phase = 1;
            if (!same && r.fo > 0) step(a);
            if (r.lx > 0) {
                if (r.twice) phase = 2;
                else if (same) phase = 4;
                return emit(a, p, r.ln, r.lh, 0, r.lx, r.twice, kFromInit, kPublish);
            }
        }
        if (phase == 2) {
            phase = same ? 4 : 1;
            return emit(a, p, r.ln, r.lh, 0, r.lx, false, kFromInit, kNothing);
        }
        if (phase == 1) {
            if (n < r.ln || (n == r.ln && h < r.lh)) {
                const int un = n, uh = h;
                step(a);
                return emit(a, p, un, uh, 0, seq_chunks(a, un, bad), false, kFromInit, kFinal);
            }
            phase = 4;
            if (r.fo > 0) return emit(a, p, r.fn, r.fh, r.fo, seq_chunks(a, r.fn, bad), false, kFromOthers, kFinal);
        }
        if (phase == 3) {
            phase = 4;
            return emit(a, p, r.fn, r.fh, r.fo, r.lx, false, kFromOthers, kNothing);
        }
        return false;
    }
};

// ... and their chunks, which the loading warp and the decays' warp walk; the latter tells the other roles.
struct Chunks {
    Pieces pieces;
    Piece p;
    int c;
    bool any;
    __device__ Chunks(const DecayPrefillArgs& a, const Range& r) : pieces(r) {
        any = pieces.next(a, p);
        c = p.c0;
    }
    __device__ __forceinline__ void next(const DecayPrefillArgs& a) {
        if (++c < p.c1) return;
        any = pieces.next(a, p);
        c = p.c0;
    }
};

// What the other roles know of a chunk.
enum ChunkFlags { kFull = 1, kFirst = 2, kLast = 4, kJoins = 8, kFinalState = 16, kLeaves = 32, kPartial = 64, kStop = 128, kInit = 256 };
struct ChunkInfo {
    int n, h, c, row0;  // row0: the chunk's first row
    int left, rows, flags, pad;  // left: rows of the sequence from this chunk on
};

// ld32 without the wait: the registers are valid after the next wait_ld().
__device__ __forceinline__ void ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ bool try_wait(uint32_t mbar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(mbar), "r"(parity)
        : "memory");
    return done;
}
__device__ __forceinline__ int gone_of(uint32_t gone) {  // the block's mark of a wait that ran out
    int x;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(x) : "r"(gone) : "memory");
    return x;
}
// The rest of a wait whose first try did not do.  When the limit is reached, or another wait of the block has run
// out, it returns all the same, with the mark set.
__device__ __noinline__ void wait_on(uint32_t mbar, uint32_t parity, uint32_t gone) {
#pragma unroll 1
    for (uint32_t it = 0; it < kWaitLimit; ++it)
        if (try_wait(mbar, parity) || gone_of(gone)) return;
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(gone), "r"(1) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ float lds_f1(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
// One box of a 3-D tensor map at (x, y, z) into L2, and one from shared memory (bulk group of the thread).
__device__ __forceinline__ void prefetch_3d(const void* map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void store_3d(const void* map, int x, int y, int z, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
// The upper halves of two fp32 values: packed, and as values.
__device__ __forceinline__ uint32_t upper(float2 x) { return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632); }
__device__ __forceinline__ float2 upper_of(float2 x) {
    return make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffff0000u), __uint_as_float(__float_as_uint(x.y) & 0xffff0000u));
}
// Four 8 x 8 blocks of 16-bit elements, transposed on the way to or from registers.
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t* r) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
// 16 lanes (rows) of 16 columns: register 2i + j of lane l is row 8j + l / 4, column 4i + l % 4.
__device__ __forceinline__ void st16x128(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Eight results from o[e] as one 16-byte word.
template <int DT>
__device__ __forceinline__ uint4 pack16(const float (&o)[32], int e) {
    return make_uint4(Elem<DT>::put2(o[e], o[e + 1]), Elem<DT>::put2(o[e + 2], o[e + 3]), Elem<DT>::put2(o[e + 4], o[e + 5]),
                      Elem<DT>::put2(o[e + 6], o[e + 7]));
}

// A row of results from tensor memory to its place: outputs of 32 bits, and chunks that a sequence ends in.
__device__ __noinline__ void store_rows(uint32_t taddr, float f, const uint8_t* to, int dt, bool there) {
    uint8_t* p = const_cast<uint8_t*>(to);
#pragma unroll 1
    for (int c = 0; c < kD; c += 16) {
        float o[16];
        ld16(taddr + c, o);
        if (there)
#pragma unroll
            for (int z = 0; z < 16; z += 4) store4_as(p, c + z, make_float4(o[z] * f, o[z + 1] * f, o[z + 2] * f, o[z + 3] * f), dt);
    }
    fence_before();
}

// 64 elements of a state, `stride` elements apart, from and to memory (all in flight together); and joined to those
// that another CTA left.
template <class T>
__device__ __forceinline__ void get_as(float* S, const T* p, size_t stride) {
    T x[64];
#pragma unroll
    for (int e = 0; e < 64; ++e) x[e] = p[e * stride];
#pragma unroll
    for (int e = 0; e < 64; ++e) S[e] = (float)x[e];
}
template <class T>
__device__ __forceinline__ void put_as(const float* S, T* p, size_t stride) {
#pragma unroll
    for (int e = 0; e < 64; ++e) p[e * stride] = (T)S[e];
}
__device__ __noinline__ void get_state(float* S, const void* from, size_t at, size_t stride, int st) {
    if (st == kStateF32) get_as(S, static_cast<const float*>(from) + at, stride);
    else if (st == kStateBF16) get_as(S, static_cast<const __nv_bfloat16*>(from) + at, stride);
    else get_as(S, static_cast<const __half*>(from) + at, stride);
}
__device__ __noinline__ void put_state(const float* S, void* to, size_t at, size_t stride, int st) {
    if (st == kStateF32) put_as(S, static_cast<float*>(to) + at, stride);
    else if (st == kStateBF16) put_as(S, static_cast<__nv_bfloat16*>(to) + at, stride);
    else put_as(S, static_cast<__half*>(to) + at, stride);
}
__device__ __noinline__ void join_state(float* S, float f, const float* from) {
    float x[64];
#pragma unroll
    for (int e = 0; e < 64; ++e) x[e] = __ldcg(from + e * 256);
#pragma unroll
    for (int e = 0; e < 64; ++e) S[e] = fmaf(f, S[e], x[e]);
}

// Q S_0's rows to the scale of the weights, as the sum that P V goes on: `cols` columns of this thread's lane.
__device__ __forceinline__ void scale_rows(uint32_t taddr, int cols, float f) {
    fence_after();
#pragma unroll 1
    for (int c = 0; c < cols; c += 32) {
        float x[32];
        ld32(taddr + c, x);
#pragma unroll
        for (int z = 0; z < 32; z += 2) {
            const float2 y = __fmul2_rn(make_float2(x[z], x[z + 1]), make_float2(f, f));
            x[z] = y.x, x[z + 1] = y.y;
        }
        st32(taddr + c, x);
    }
    wait_st();
    fence_before();
}

// The power of two, at most 2^60, that takes x into [2^13, 2^14); 1 for zero, infinities and NaN.
__device__ __forceinline__ float range_scale(float x) {
    const int e = (int)(__float_as_uint(x) >> 23) & 255;
    return x == 0.f || e == 255 ? 1.f : __uint_as_float((uint32_t)min(max(267 - e, 2), 187) << 23);
}
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }

template <int DT>
__global__ void __launch_bounds__(kPreDecayThreads, 1)
    decay_prefill_kernel(const __grid_constant__ DecayMaps maps, const __grid_constant__ DecayPrefillArgs a) {
    using E = Elem<DT>;
    constexpr bool kF16 = DT == KDA_F16;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* ctrl = reinterpret_cast<int*>(sm + DS_CTRL);  // 0 tensor memory, 1 waits that ran out, 2.. the range, 8 the first unit's place
    volatile long long* scan = reinterpret_cast<long long*>(sm + DS_SCAN);
    auto bar = [&](int i) { return sb + DS_BAR + 8 * i; };
    const bool cut = a.flags != nullptr;

    if (tid == 0) {
        if (a.T > 0) {
            prefetch_map(&maps.q);
            prefetch_map(&maps.k);
            prefetch_map(&maps.v);
        }
        ctrl[1] = 0;
    }
    // ---- this CTA's range of chunks
    Range rg;
    int64_t total = 0, unit_at = 0;  // the places of all units (a place a chunk, then kUnitChunks); the first unit's first place
    int ctas = 1;
    if (!cut) {
        int bad;
        const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H, c = seq_chunks(a, n, bad);
        rg = Range{n, h, 0, h + 1 < a.H ? n : n + 1, h + 1 < a.H ? h + 1 : 0, 0, false};
        if (tid == 0 && h == 0 && bad) report(a.dev_status, bad);
        if (c == 0) return;
    } else {
        // Inclusive sums over 512 values, or over 32 that every warp has alike.
        const bool few = a.N <= 32;
        const int me = few ? lane : tid, width = few ? 32 : kPreDecayThreads;
        auto sums = [&](int64_t x, int64_t& sum) {
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            sum = __shfl_sync(~0u, x, 31);
            if (few) return x;
            __syncthreads();
            if (lane == 31) scan[warp] = x;
            __syncthreads();
            int64_t off = 0;
            sum = 0;
            for (int w = 0; w < kPreDecayThreads / 32; ++w) {
                const int64_t y = scan[w];
                if (w < warp) off += y;
                sum += y;
            }
            return x + off;
        };
        const int64_t one = a.N <= 65536 ? 1ll << 40 : 0;  // the units' number, in the upper bits (places stay below 2^39 then)
        int64_t mine = 0;
        for (int n = me; n < a.N; n += width) {
            int bad;
            const int c = seq_chunks(a, n, bad);
            mine += c ? c + kUnitChunks + one : 0;
            if (bad && blockIdx.x == 0 && tid < width) report(a.dev_status, bad);
        }
        sums(mine, total);
        const int64_t units = one ? (total >> 40) * a.H : 0;
        total = (one ? total & (one - 1) : total) * a.H;
        const int64_t least = total < kShortUnit * units ? units : (total + kCutChunks - 1) / kCutChunks;
        ctas = (int)min((int64_t)gridDim.x, least);
        if ((int)blockIdx.x >= ctas) return;
        if (tid == 0) {
            ctrl[5] = a.N;  // the last CTA's end
            ctrl[6] = ctrl[7] = ctrl[10] = 0;
        }
        __syncthreads();
        int64_t before = 0;
        for (int base = 0; base < a.N; base += width) {
            const int n = base + me;
            int bad;
            const int chunks = n < a.N ? seq_chunks(a, n, bad) : 0, c = chunks ? chunks + kUnitChunks : 0;
            int64_t sum;
            const int64_t end = (before + sums(c, sum)) * a.H, begin = end - (int64_t)c * a.H;
            before += sum;
            for (int e = 0; e < 2; ++e) {
                const int64_t x = total * (blockIdx.x + e) / ctas;
                if (c && x >= begin && x < end && tid < width) {
                    const int64_t h = (x - begin) / c, unit = begin + h * c;
                    const bool past = x - unit >= chunks;  // the next unit
                    ctrl[2 + 3 * e] = n;
                    ctrl[3 + 3 * e] = (int)h + past;
                    ctrl[4 + 3 * e] = past ? 0 : (int)(x - unit);
                    if (e == 0) *reinterpret_cast<volatile long long*>(sm + DS_CTRL + 32) = unit;
                    else ctrl[10] = !past && total * (blockIdx.x + 2) / ctas < unit + chunks;
                }
            }
        }
        __syncthreads();
        rg = Range{ctrl[2], ctrl[3], ctrl[4], ctrl[5], ctrl[6], ctrl[7], ctrl[10] != 0};
        auto carry = [&](int& n, int& h) {  // from behind the last head to the next sequence
            int bad;
            if (h < a.H) return;
            h = 0;
            do ++n;
            while (n < a.N && seq_chunks(a, n, bad) == 0);
        };
        carry(rg.fn, rg.fh);
        carry(rg.ln, rg.lh);
        unit_at = *reinterpret_cast<volatile long long*>(sm + DS_CTRL + 32);
    }
    if (tid < B_COUNT) {
        int count = 1;
        if (tid == B_P || tid == B_SCALED || tid == B_OFREE) count = 4;      // warps
        if (tid == B_SPLIT || tid == B_SPLIT + 1 || tid == B_S || tid == B_MEET) count = 8;
        if (tid == B_GFREE || tid == B_GFREE + 1) count = 13;
        if (tid == B_FREE || tid == B_FREE + 1) count = 5;  // four warps and a commit
        if (tid == B_TAKEN || tid == B_TAKEN + 1) count = 8;
        mbar_init(bar(tid), count);
    }
    if (warp == 1) tmem_alloc(sb + DS_CTRL, 512);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = ctrl[0];

    // A wait that runs out marks the block: its roles then end with the chunk they are at, and nothing is stored any
    // more.  (That, and what is rare, stays out of line: the roles share an instruction cache.)
    const uint32_t gone = sb + DS_CTRL + 4;
    auto wait = [&](int b, uint32_t parity) {
        if (!try_wait(bar(b), parity)) wait_on(bar(b), parity, gone);
    };
    auto dead = [&] { return __any_sync(~0u, gone_of(gone)); };
    auto arrive = [&](int b) {  // of a warp
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b));
    };
    const uint32_t g_d = sb + DS_G, g_tot = sb + DS_TOT;  // a stage: D [128], e^-D [128]; totals [4], the chunk's decay, its ChunkInfo, e^ of the totals behind each block [4]
    auto info_of = [&](uint32_t st) {
        const uint4 x = lds128(g_tot + 80 * st + 32), y = lds128(g_tot + 80 * st + 48);
        return ChunkInfo{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, 0};
    };

    if (warp == 0) {
        // ================================================================ loads
        uint32_t it = 0, m = 0;
        for (Chunks ch(a, rg); ch.any && !dead(); ch.next(a), ++it) {
            const uint32_t st = it & 1;
            if ((int)blockIdx.x == a.give_up_cta && (int)it == a.give_up_load) {
                ctrl[1] = 1;
                break;
            }
            const int row = ch.p.row0 + ch.c * kDecayChunk, h = ch.p.h, hk = h / a.group;
            if (it >= 2) wait(B_FREE + st, ((it >> 1) - 1) & 1);
            auto load = [&](uint32_t dst, const CUtensorMap* map, int head, int b) {
                if (lane != 0) return;
                if (ch.p.rows == 0) {  // an empty sequence's one chunk: its keys and values are cleared, its scores not used
                    mbar_arrive(bar(b));
                    return;
                }
                mbar_expect_tx(bar(b), kTile);
                tma_load_3d(sb + dst, map, 0, head, row, bar(b));
                tma_load_3d(sb + dst + kTile / 2, map, 64, head, row, bar(b));
            };
            load(DS_K + st * kTile, &maps.k, hk * a.hk, B_KF + st);
            load(DS_V + st * kTile, &maps.v, h * a.hv, B_VF + st);
            if (!ch.p.state_only) {
                if (m > 0) wait(B_QS, (m - 1) & 1);
                load(DS_Q, &maps.q, hk * a.hq, B_QF);
                ++m;
            }
            if (ch.c == ch.p.c0 && ch.p.start == kFromInit && a.init_slot && lane == 0) {
                const int src = a.init_slot[ch.p.n];
                if (src >= 0) bulk_prefetch_l2(static_cast<const uint8_t*>(a.pool) + state_elem(src, a.H, h) * state_bytes(a.st), kD * kD * state_bytes(a.st));
            }
            // the next chunk into L2: its loads wait for their buffers (Q's for this chunk's Q S), and from HBM they
            // took 4400 cycles then
            if (ch.c + 1 < ch.p.c1 && lane < (ch.p.state_only ? 4 : 6)) {
                const int which = lane >> 1, head = which == 0 ? hk * a.hk : which == 1 ? h * a.hv : hk * a.hq;
                prefetch_3d(which == 0 ? &maps.k : which == 1 ? &maps.v : &maps.q, 64 * (lane & 1), head, row + kDecayChunk);
            }
        }
    } else if (warp == 1) {
        // ================================================================ products
        // the whole warp runs this, one lane issues (umma.cuh, mma_by)
        const uint32_t lead = elect_lane();
        const uint32_t sb4 = (sb & 0x3ffffu) >> 4, t4 = kTile >> 4;
        const uint32_t tm = __shfl_sync(~0u, tmem, 0);
        const uint32_t i_qk = idesc_16(kF16, 128, 128, false, false, false);
        const uint32_t i_tv = idesc_16(kF16, 128, 128, false, true, false);  // B with its rows along N
        const uint32_t i_tt = idesc_16(kF16, 128, 128, true, true, false);   // and A with its along M
        // descriptors of step s: rows of channels, and rows of tokens (a step's 16 tokens behind one another)
        auto along_k = [&](uint32_t at4, uint32_t s) { return desc4(at4 + (s >> 2) * 1024 + (s & 3) * 2, 16, 1024); };
        auto along_mn = [&](uint32_t at4, uint32_t s) { return desc4(at4 + 128 * s, kTile / 2, 1024); };
        const uint32_t q4 = sb4 + DS_Q / 16, s4 = sb4 + DS_S / 16, lo4 = sb4 + DS_LO / 16;
        int flags = 0;  // of chunk it
        uint32_t m = 0;
        for (uint32_t it = ~0u;; ++it) {
            // Chunk `it` in the order in which operands come, and the next chunk's scores (over this one's weights, so
            // behind P V).  The waits suspend the warp: a loop that tested all barriers in turn took so many issue slots
            // from the three warps beside it that every role waited for those.
            const uint32_t st = it & 1, sn = st ^ 1;
            const bool full = flags & kFull;
            const uint32_t v4 = sb4 + DS_V / 16 + st * t4;
            if (it != ~0u) {
                wait(B_VF + st, (it >> 1) & 1);
#pragma unroll 1
                for (uint32_t i = 0; i < 2; ++i) {  // 32 of each 64 tokens
                    wait(B_SPLIT + i, it & 1);
                    fence_after();
                    // the smallest part first: what a sum of products loses goes by its size so far
                    if constexpr (!kF16) {
#pragma unroll
                        for (uint32_t x = 0; x < 4; ++x) {
                            const uint32_t s = 2 * i + (x & 1) + 4 * (x >> 1);
                            mma_by(lead, tm + DT_KV, along_mn(lo4, s), along_mn(v4, s), i_tt, i | x);
                        }
                    }
#pragma unroll 1
                    for (uint32_t part = 0; part < 2; ++part)
#pragma unroll
                        for (uint32_t x = 0; x < 4; ++x) {
                            const uint32_t s = 2 * i + (x & 1) + 4 * (x >> 1);
                            mma_ta_by(lead, tm + DT_KV, tm + (part ? DT_K1 : DT_K2) + 8 * s, along_mn(v4, s), i_tv,
                                      !kF16 || part > 0 || (i | x));
                        }
                }
                commit_by(lead, bar(B_KV));
            }
            if (full) {
                wait(B_S, m & 1);
                if (m > 0) wait(B_OFREE, (m - 1) & 1);
                fence_after();
#pragma unroll
                for (uint32_t s = 0; s < 8; ++s) mma_by(lead, tm + DT_O, along_k(q4, s), along_mn(s4, s), i_tv, s);
                commit_by(lead, bar(B_QS));
                wait(B_P, m & 1);
                wait(B_SCALED, m & 1);
                fence_after();
#pragma unroll
                for (uint32_t s = 0; s < 8; ++s) mma_ta_by(lead, tm + DT_O, tm + DT_SC + 8 * s, along_mn(v4, s), i_tv, 1);
                commit_by(lead, bar(B_O));
                ++m;
            }
            if (it != ~0u) commit_by(lead, bar(B_FREE + st));  // keys and values have had all their products
            wait(B_GF + sn, ((it + 1) >> 1) & 1);
            flags = __shfl_sync(~0u, info_of(sn).flags, 0);
            if ((flags & kStop) || dead()) break;
            arrive(B_GFREE + sn);
            if (flags & kFull) {
                wait(B_QF, m & 1);
                wait(B_KF + sn, ((it + 1) >> 1) & 1);
#pragma unroll
                for (uint32_t s = 0; s < 8; ++s)
                    mma_by(lead, tm + DT_SC, along_k(q4, s), along_k(sb4 + DS_K / 16 + sn * t4, s), i_qk, s);
                commit_by(lead, bar(B_QK));
            }
        }
        commit_by(lead, bar(B_DRAIN));
        for (uint32_t polls = 0; polls < kWaitLimit && !try_wait(bar(B_DRAIN), 0); ++polls) {
        }
    } else if (warp < 4) {
        // ================================================================ decays: lane l has tokens 4l .. 4l + 3
        // two warps in turns, each with the next log decays it needs in flight
        Chunks ch(a, rg);
        if (warp == 3 && ch.any) ch.next(a);
        float ahead[4];
        auto ask = [&] {
            const int first = ch.c * kDecayChunk + 4 * lane;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                ahead[e] = ch.any && first + e < ch.p.rows
                               ? log_decay_of(a.head_decay, a.log_decay, (int64_t)ch.p.row0 + first + e, a.H, ch.p.h)
                               : 0.f;
        };
        ask();
        for (uint32_t it = warp & 1; !dead(); it += 2) {
            const uint32_t st = it & 1;
            const bool any = ch.any;
            const int before = ch.c * kDecayChunk;
            const Piece& p = ch.p;
            const int flags = !any ? kStop
                                   : (p.state_only ? 0 : kFull) | (ch.c == p.c0 ? kFirst : 0) | (ch.c + 1 == p.c1 ? kLast : 0) |
                                         (p.start == kFromOthers ? kJoins : 0) | (p.start == kFromInit ? kInit : 0) | (p.end == kFinal ? kFinalState : 0) |
                                         (p.end == kPublish ? kLeaves : 0) | (p.rows - before < kDecayChunk ? kPartial : 0);
            const int4 info1 = make_int4(p.n, p.h, ch.c, p.row0 + before), info2 = make_int4(p.rows - before, p.rows, flags, 0);
            double g[4], y0 = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = y0 += (double)ahead[e] * 1.4426950408889634;
            if (any) ch.next(a);
            if (ch.any) ch.next(a);
            ask();
            double x = g[3];
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            const double end = __shfl_sync(~0u, x, lane | 7), all = __shfl_sync(~0u, x, 31);
            const double last = __shfl_sync(~0u, x, max((lane & 24) - 1, 0));
            const double excl = x - g[3] - end;
            const float4 d = make_float4((float)(excl + g[0]), (float)(excl + g[1]), (float)(excl + g[2]), (float)(x - end));
            // the chunk's decay 2^all, once rounded (it multiplies the state chunk after chunk, and an error alike in each
            // would grow): 2^n times the exponential series of the rest, |rest ln 2| <= 0.35
            const double n = rint(fmax(all, -1000.0)), y = (all - n) * 0.6931471805599453;
            double z = 1.0;
#pragma unroll
            for (int k = 10; k > 0; --k) z = fma(z * y, 1.0 / k, 1.0);
            const float chunk = n < -126.0 ? 0.f : (float)z * __int_as_float(((int)n + 127) << 23);
            if (it >= 2) wait(B_GFREE + st, ((it >> 1) - 1) & 1);
            {
                const uint32_t at = DS_G + st * 1024 + 16 * lane;
                *reinterpret_cast<float4*>(sm + at) = d;
                *reinterpret_cast<float4*>(sm + at + 512) = make_float4(ex2(-d.x), ex2(-d.y), ex2(-d.z), ex2(-d.w));
                float* tot = reinterpret_cast<float*>(sm + DS_TOT + st * 80);
                if ((lane & 7) == 0) {
                    tot[lane >> 3] = (float)(end - (lane < 8 ? 0.0 : last));
                    tot[16 + (lane >> 3)] = ex2((float)(all - end));
                }
                if (lane == 0) {
                    tot[4] = isnan(all) ? (float)all : chunk;
                    *reinterpret_cast<int4*>(tot + 8) = info1;
                    *reinterpret_cast<int4*>(tot + 12) = info2;
                }
            }
            arrive(B_GF + st);
            if (!any) break;
        }
    } else if (warp >= 4 && warp < 8) {
        // ================================================================ weights and results: a thread has a row
        const int w = warp & 3, row = 32 * w + lane;
        const uint32_t tl = tmem + ((uint32_t)(w * 32) << 16);
        const float scale = a.scale;
        uint32_t m = 0;
        int owed = -1;  // the stage whose stored results have not been waited for
        auto give_back = [&] {
            if (owed < 0) return;
            if (lane == 0) bulk_wait_read_all();
            arrive(B_FREE + owed);
            owed = -1;
        };
        for (uint32_t it = 0;; ++it) {
            const uint32_t st = it & 1;
            wait(B_GF + st, (it >> 1) & 1);
            const ChunkInfo ch = info_of(st);
            if ((ch.flags & kStop) || dead()) break;
            if (!(ch.flags & kFull)) {
                arrive(B_GFREE + st);
                give_back();
                // not before the stage's last chunk has had its products: an early arrival would count for that one
                if (it >= 2) wait(B_FREE + st, ((it >> 1) - 1) & 1);
                arrive(B_FREE + st);
                continue;
            }
            const uint32_t gd = g_d + st * 1024;
            const float4 tot4 = lds_f4(g_tot + st * 80);
            const float tot[4] = {tot4.x, tot4.y, tot4.z, tot4.w};
            const float d = lds_f1(gd + 4 * row);
            wait(B_QK, m & 1);
            fence_after();
            float ps = 1.f, lps = 0.f;  // fp16: the row's scale
            if constexpr (kF16) {
                float mx = 0.f, my = 0.f;
#pragma unroll 1
                for (int b = 0; b < w; ++b) {
                    float s[32];
                    ld32(tl + DT_SC + 32 * b, s);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        mx = fmaxf(fmaxf(mx, fabsf(s[e])), fabsf(s[e + 1]));
                        my = fmaxf(fmaxf(my, fabsf(s[e + 2])), fabsf(s[e + 3]));
                    }
                }
                float s[32];
                ld32(tl + DT_SC + 32 * w, s);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    mx = e <= lane ? fmaxf(mx, fabsf(s[e])) : mx;
                    my = e + 1 <= lane ? fmaxf(my, fabsf(s[e + 1])) : my;
                }
                ps = range_scale(fmaxf(mx, my));
                lps = (float)((int)(__float_as_uint(ps) >> 23) - 127);
            }
            float gi = d;  // G_i
#pragma unroll
            for (int x = 0; x < 4; ++x) gi += x <= w ? tot[x] : 0.f;
            // Weights and Q S_0 are summed at the scale 2^-ref, ref = max(G_i, -60) (bf16: weights are 2^60 at most), so
            // that Q S_0 is taken as it is unless the row's decay is below 2^-60.  fp16 weights take the row's own scale.
            const float ref = kF16 ? -lps : fmaxf(gi, -60.f);
            // blocks before the diagonal one, that one, then zeros; a block's scores are asked for ahead of its turn
            const float dr = d - ref;
            uint32_t ahead[32];
            ld32_issue(tl + DT_SC, ahead);
#pragma unroll 1
            for (int b = 0; b <= w; ++b) {
                float s[32];
                wait_ld();
#pragma unroll
                for (int x = 0; x < 32; ++x) s[x] = __uint_as_float(ahead[x]);
                if (b < w) ld32_issue(tl + DT_SC + 32 * (b + 1), ahead);
                uint32_t p[16];
                if (b < w) {
                    float e = d - ref;
#pragma unroll
                    for (int x = 1; x < 4; ++x) e += x > b && x <= w ? tot[x] : 0.f;
                    const float f = ex2(e);
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {
                        const float4 c = lds_f4(gd + 512 + 4 * (32 * b + x));
                        const float4 y = f4_mul(f4_mul(make_float4(s[x], s[x + 1], s[x + 2], s[x + 3]), c), make_float4(f, f, f, f));
                        p[x / 2] = E::put2(y.x, y.y);
                        p[x / 2 + 1] = E::put2(y.z, y.w);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {
                        const float4 c = lds_f4(gd + 4 * (32 * b + x));
                        const float cc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) s[x + y] = x + y <= lane ? s[x + y] * ex2(dr - cc[y]) : 0.f;
                        p[x / 2] = E::put2(s[x], s[x + 1]);
                        p[x / 2 + 1] = E::put2(s[x + 2], s[x + 3]);
                    }
                }
                // (over scores of this block and, for the second, the first: both have been read)
                st16u(tl + DT_SC + 16 * b, p);
            }
            for (int b = w + 1; b < 4; ++b) {
                uint32_t p[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) p[x] = 0;
                st16u(tl + DT_SC + 16 * b, p);
            }
            wait_st();
            fence_before();
            arrive(B_P);
            give_back();
            arrive(B_GFREE + st);
            float fp = scale;  // the sum's factor
            if constexpr (kF16) {
                wait(B_QS, m & 1);
                scale_rows(tl + DT_O, 128, ps * ex2(gi) * pow2_inverse(lds_f1(sb + DS_SCALE + 4 * (m & 1))));
                fp *= pow2_inverse(ps);
            } else {
                if (__any_sync(~0u, !(gi >= -60.f))) {
                    wait(B_QS, m & 1);
                    scale_rows(tl + DT_O, 128, ex2(gi - ref));
                }
                fp *= ex2(ref);
            }
            arrive(B_SCALED);
            wait(B_O, m & 1);
            fence_after();
            const bool boxes = a.boxes && !(ch.flags & kPartial);
            if (boxes) {
                wait(B_TAKEN + st, (it >> 1) & 1);
                const uint32_t stage = sb + DS_K + st * kTile;  // of these keys
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    float o[32];
                    ld32(tl + DT_O + 32 * b, o);
#pragma unroll
                    for (int z = 0; z < 32; z += 2) {
                        const float2 y = __fmul2_rn(make_float2(o[z], o[z + 1]), make_float2(fp, fp));
                        o[z] = y.x, o[z + 1] = y.y;
                    }
                    const uint32_t to = stage + (b >> 1) * (kTile / 2) + row * 128, c = 4 * (b & 1);
#pragma unroll
                    for (int z = 0; z < 4; ++z) sts128(to + (((c + z) ^ (row & 7)) << 4), pack16<DT>(o, 8 * z));
                }
                fence_before();
                fence_async_smem();
                arrive(B_OFREE);
                if (!dead() && lane == 0) {
                    for (int x = 0; x < 2; ++x)
                        store_3d(&maps.out, 64 * x, ch.h * a.ho, ch.row0 + 32 * w, stage + x * (kTile / 2) + 32 * w * 128);
                    bulk_commit();
                }
                owed = (int)st;
            } else {
                arrive(B_FREE + st);
                const int64_t o_at = ((int64_t)ch.row0 + row) * a.out.rs + ch.h * a.out.hs;
                store_rows(tl + DT_O, fp, reinterpret_cast<const uint8_t*>(a.out.base) + o_at * dtype_bytes(a.out_dt), a.out_dt,
                           !dead() && row < ch.left);
                arrive(B_OFREE);
            }
            ++m;
        }
        if (lane == 0) bulk_wait_all();
    } else if (warp >= 8) {
        // ================================================================ keys and state
        // A thread has key channel `key` of the state, value channels 64 half .. 64 half + 63; of the keys' split its
        // warp has 32 channels of 64 tokens.
        const int t = tid - 256, half = t >> 7, key = t & 127;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float S[64], decay = 1.f;
        uint32_t it = 0, m = 0, met = 0;
        // the eight warps wait for one another, with a limit as everywhere
        auto meet = [&] {
            arrive(B_MEET);
            wait(B_MEET, met++ & 1);
        };
        // this thread's elements of a state in memory, whose rows are value channels
        auto elems = [&](int64_t slot, int h) { return state_elem(slot, a.H, h) + (size_t)(64 * half) * kD + key; };
        auto store_state = [&](void* to, size_t at, size_t stride, int st) {
            if (st == kStateF32) {
                float* p = static_cast<float*>(to) + at;
                if (!dead())
#pragma unroll
                    for (int e = 0; e < 64; ++e) p[e * stride] = S[e];
                return;
            }
            float x[64];  // (the registers themselves have no address)
#pragma unroll
            for (int e = 0; e < 64; ++e) x[e] = S[e];
            if (!dead()) put_state(x, to, at, stride, st);
        };
        // ldmatrix of 8 x 8 blocks, transposed: block j of four has channels 8 (j & 1) .. and tokens 8 (j >> 1) .., its
        // row r lies at token r; the other block of 64 channels 16 KiB on
        const int blk = lane >> 3, chunk16 = (32 * (warp & 3) & 63) / 8 + (blk & 1);
        const uint32_t k_row = (uint32_t)((warp & 3) >> 1) * (kTile / 2) + (64 * half + 8 * (blk >> 1) + (lane & 7)) * 128;
        for (;; ++it) {
            const uint32_t st = it & 1;
            wait(B_GF + st, (it >> 1) & 1);
            const ChunkInfo p = info_of(st);
            if ((p.flags & kStop) || dead()) break;
            const bool full = p.flags & kFull;
            const float ac = lds_f1(g_tot + st * 80 + 16);
            wait(B_KF + st, (it >> 1) & 1);
            if (p.left < kDecayChunk) {
                // rows past the sequence have a weight of zero, and so has to be the value
                wait(B_VF + st, (it >> 1) & 1);
                for (int x = max(p.left, 0) * 8 + t; x < 1024; x += 256) {
                    sts128(sb + DS_V + st * kTile + 16 * x, make_uint4(0, 0, 0, 0));
                    sts128(sb + DS_V + st * kTile + kTile / 2 + 16 * x, make_uint4(0, 0, 0, 0));
                }
            }
            // ---- K~: 32 tokens (a block of the decays) at a time, so that the second's split runs under the first's products
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int token = 64 * half + 32 * i + 2 * (lane & 3);  // and the next one, of each group of 8
                const float after = lds_f1(g_tot + st * 80 + 64 + 4 * (2 * half + i));
                float2 f[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];"
                                 : "=f"(f[g].x), "=f"(f[g].y)
                                 : "r"(g_d + st * 1024 + 512 + 4 * (token + 8 * g)));
                    f[g] = __fmul2_rn(f[g], make_float2(after, after));
                }
#pragma unroll 1
                for (int lh = 0; lh < 2; ++lh) {  // 16 channels
                    const uint32_t at = k_row + 4096 * i + (((chunk16 + 2 * lh) ^ (lane & 7)) << 4);
                    uint32_t k[8], mid[8], lo[8];
                    ldsm4t(sb + DS_K + st * kTile + at, k);
                    ldsm4t(sb + DS_K + st * kTile + at + 2048, k + 4);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const float2 minus = make_float2(-1.f, -1.f);
                        float2 y = __fmul2_rn(E::get2(k[x]), f[x >> 1]);
                        if (p.left < kDecayChunk) {  // whatever lies past the sequence
                            if (token + 8 * (x >> 1) >= p.left) y.x = 0.f;
                            if (token + 8 * (x >> 1) + 1 >= p.left) y.y = 0.f;
                        }
                        if constexpr (kF16) {
                            k[x] = E::put2(y.x, y.y);
                            y = __ffma2_rn(E::get2(k[x]), minus, y);
                            mid[x] = E::put2(y.x, y.y);
                        } else {  // three times the upper 8 bits of what is left: nothing is
                            k[x] = upper(y);
                            y = __ffma2_rn(upper_of(y), minus, y);
                            mid[x] = upper(y);
                            y = __ffma2_rn(upper_of(y), minus, y);
                            lo[x] = upper(y);
                        }
                    }
                    const uint32_t to = tl + ((uint32_t)(16 * lh) << 16) + 32 * half + 16 * i;
                    st16x128(to + DT_K1, k);
                    st16x128(to + DT_K2, mid);
                    if constexpr (!kF16) {
                        stsm4t(sb + DS_LO + at, lo);
                        stsm4t(sb + DS_LO + at + 2048, lo + 4);
                    }
                }
                wait_st();
                fence_before();
                fence_async_smem();
                arrive(B_SPLIT + i);
            }
            arrive(B_TAKEN + st);
            arrive(B_GFREE + st);
            // ---- the state before this chunk, under the products
            if (p.flags & kFirst) {
#pragma unroll
                for (int e = 0; e < 64; ++e) S[e] = 0.f;
                decay = 1.f;
                if (p.flags & kInit) {
                    const int src = a.init_slot ? a.init_slot[p.n] : -1;
                    // The second pass over a unit's beginning comes after its state was left: its last CTA may be done by
                    // then and have written the very slot.  So that pass starts from a copy.
                    const size_t copy = (size_t)(kDecayCtas + blockIdx.x) * (kD * kD) + t;
                    const bool second = full && !(p.flags & (kFinalState | kLeaves));
                    if (src >= 0 && (second || a.st == kStateF32)) {
                        const float* from = second ? a.states + copy : static_cast<const float*>(a.pool) + elems(src, p.h);
                        const size_t stride = second ? 256 : kD;
#pragma unroll
                        for (int e = 0; e < 64; ++e) S[e] = from[e * stride];
                    } else if (src >= 0) {
                        float x[64];  // (the registers themselves have no address)
                        get_state(x, a.pool, elems(src, p.h), kD, a.st);
#pragma unroll
                        for (int e = 0; e < 64; ++e) S[e] = x[e];
                    }
                    if (src >= 0 && !full) store_state(a.states, copy, 256, kStateF32);
                    if (p.h == 0 && t == 0 && full)
                        for (int y = 0; y < a.M; ++y) {
                            const int c = a.track_idx[(int64_t)p.n * a.M + y];
                            if (c < -1 || c >= (p.rows + kDecayChunk - 1) / kDecayChunk) report(a.dev_status, KDA_DEV_BAD_TRACK);
                        }
                } else if (p.flags & kJoins) {
                    float x[64];
#pragma unroll
                    for (int e = 0; e < 64; ++e) x[e] = 0.f;
                    // the CTA with the unit's beginning left a state, those after it their ranges' own; a lane waits for each
                    for (int j0 = (int)(((unit_at + 1) * ctas - 1) / total); j0 < (int)blockIdx.x; j0 += 32) {
                        const int j = min(j0 + lane, (int)blockIdx.x - 1);
                        uint32_t set = 0;
#pragma unroll 1
                        for (uint32_t polls = 0; polls < kFlagLimit && !set && !gone_of(gone); ++polls) {
                            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(set) : "l"(a.flags + j) : "memory");
                            if (!set) __nanosleep(64);
                        }
                        const float f = set ? *(volatile float*)(a.decays + j) : 0.f;
                        if (!__all_sync(~0u, set)) {
                            ctrl[1] = 1;
                            break;
                        }
                        // a lane reads states whose flags others acquired: the vote and the shuffles order no memory
                        __syncwarp();
                        const int n = min((int)blockIdx.x - j0, 32);
                        for (int y = 0; y < n; ++y)
                            join_state(x, __shfl_sync(~0u, f, y), a.states + (size_t)(j0 + y) * (kD * kD) + t);
                    }
#pragma unroll
                    for (int e = 0; e < 64; ++e) S[e] = x[e];
                }
            }
            if (full) {
                if (a.M > 0 && p.rows > 0) {
                    for (int base = 0; base < a.M; base += 32) {
                        const int x = base + lane < a.M ? a.track_idx[(int64_t)p.n * a.M + base + lane] : -1;
                        for (uint32_t hit = __ballot_sync(~0u, x == p.c); hit; hit &= hit - 1)
                            store_state(a.track, elems((int64_t)p.n * a.M + base + __ffs(hit) - 1, p.h), kD, a.st);
                    }
                }
                float ss = 1.f;
                if constexpr (kF16) {
                    float mx = 0.f;
#pragma unroll
                    for (int e = 0; e < 64; ++e) mx = fmaxf(mx, fabsf(S[e]));
                    const uint32_t wm = __reduce_max_sync(~0u, __float_as_uint(mx));
                    float* maxima = reinterpret_cast<float*>(sm + DS_MAX) + 8 * (m & 1);  // the other eight may still be read
                    if (lane == 0) maxima[warp - 8] = __uint_as_float(wm);
                    meet();
                    mx = maxima[0];
#pragma unroll
                    for (int x = 1; x < 8; ++x) mx = fmaxf(mx, maxima[x]);
                    ss = range_scale(mx);
                    if (t == 0) *reinterpret_cast<float*>(sm + DS_SCALE + 4 * (m & 1)) = ss;
                }
                if (m > 0) wait(B_QS, (m - 1) & 1);  // the last operand has been read
#pragma unroll
                    for (int e = 0; e < 64; e += 8) {
                        uint4 x;
                        x.x = E::put2(S[e] * ss, S[e + 1] * ss);
                        x.y = E::put2(S[e + 2] * ss, S[e + 3] * ss);
                        x.z = E::put2(S[e + 4] * ss, S[e + 5] * ss);
                        x.w = E::put2(S[e + 6] * ss, S[e + 7] * ss);
                        sts128(sb + DS_S + half * (kTile / 2) + key * 128 + (((e >> 3) ^ (key & 7)) << 4), x);
                    }
                fence_async_smem();
                arrive(B_S);
                ++m;
            }
            wait(B_KV, it & 1);
            fence_after();
            decay *= ac;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float x[32];
                ld32(tl + DT_KV + 64 * half + 32 * b, x);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 y = __ffma2_rn(make_float2(ac, ac), make_float2(S[32 * b + e], S[32 * b + e + 1]), make_float2(x[e], x[e + 1]));
                    S[32 * b + e] = y.x, S[32 * b + e + 1] = y.y;
                }
            }
            fence_before();
            if (!(p.flags & kLast)) continue;
            if (p.flags & kFinalState) {
                const int dst = a.final_slot ? a.final_slot[p.n] : -1;
                if (dst >= 0) store_state(a.pool, elems(dst, p.h), kD, a.st);
            } else if (p.flags & kLeaves) {
                store_state(a.states, (size_t)blockIdx.x * (kD * kD) + t, 256, kStateF32);
                if (t == 0) a.decays[blockIdx.x] = decay;
                __threadfence();
                meet();
                if (t == 0 && !gone_of(gone))
                    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(a.flags + blockIdx.x), "r"(1u) : "memory");
            }
        }
    }
    fence_before();
    __syncthreads();
    // Every load was waited for by a role that is done.  After a wait that ran out that does not hold: a bounded
    // wait on a barrier that nothing arrives on (about a second) lets them land.
    if (ctrl[1] && warp == 0) {
        for (uint32_t polls = 0; polls < kWaitLimit && !try_wait(bar(B_NEVER), 0); ++polls) {
        }
        if (lane == 0) report(a.dev_status, KDA_DEV_TIMEOUT);
        __syncwarp();
    }
    __syncthreads();
    fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Tensor map over rows of heads: (channel, head, row), one box 64 channels of one head.
bool chunk_map(CUtensorMap* map, kda_dtype dt, const LatentRows& r, int H, int T, int rows) {
    // a dimension that is not stepped along (one head or row, or heads that share a row) has size 1 and any legal stride
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)(r.hs ? H : 1), (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)(r.hs ? r.hs : kD) * 2, (cuuint64_t)(r.rs ? r.rs : kD) * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    return encode_16bit(map, dt, 3, r.base, dims, strides, box);
}

// Bytes of a cut launch's workspace: flags, decays, states left and initial states kept; none for prompts that no cut helps.
bool may_cut(int32_t T_tot) { return T_tot > kDecayChunk * kCutChunks; }
constexpr size_t kCutBytes = 2 * 4 * kDecayCtas + (size_t)2 * kDecayCtas * kD * kD * 4;

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_decay_prefill_workspace_size(int32_t T_tot, int32_t N, int32_t H) {
    return may_cut(T_tot) && N > 0 && H > 0 ? kCutBytes : 16;
}

namespace kda {
namespace {

// Both entry points; give_up_cta < 0 for the call itself.
kda_status prefill_call(
    const kda_rows_desc* q, const kda_rows_desc* k, const kda_rows_desc* v,
    kda_dtype in_dtype, const float* head_decay, const float* log_decay, const int32_t* cu_seqlens, int32_t N, int32_t T_tot,
    int32_t H, int32_t Hk, int32_t dk, int32_t dv, float scale, uint32_t flags, void* state_pool, int64_t P,
    const int32_t* init_slot, const int32_t* final_slot, const int32_t* track_chunk_idx, int32_t M, void* track_state,
    const kda_rows_desc* out, kda_dtype out_dtype, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream, int32_t give_up_cta,
    int32_t give_up_load) {
    KDA_REQUIRE(N >= 0 && T_tot >= 0 && H > 0 && Hk > 0 && P >= 0 && M >= 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(H % Hk == 0 && isfinite(scale), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(dk == kD && dv == kD, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((in_dtype == KDA_BF16 || in_dtype == KDA_F16) && any_dtype_ok(out_dtype), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((flags & ~(KDA_STATE_BF16 | KDA_STATE_F16)) == 0 && state_flags_ok(flags), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(T_tot < (1 << 30) && (int64_t)N * H < (1 << 27), KDA_ERR_UNSUPPORTED);
    if (N == 0) return KDA_OK;
    // without rows there is nothing to place, and states are passed on
    KDA_REQUIRE(T_tot == 0 || (rows_ok(q) && rows_ok(k) && rows_ok(v) && rows_ok(out)), KDA_ERR_INVALID_ARG);
    if (T_tot > 0)
        for (const kda_rows_desc* d : {q, k, v})
            KDA_REQUIRE((d->row_stride > 0 || T_tot == 1) && d->row_stride >= 0 && d->head_stride >= 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(cu_seqlens, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(state_pool || (!init_slot && !final_slot), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(M == 0 || (track_chunk_idx && track_state), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(decays_ok(head_decay, log_decay), KDA_ERR_INVALID_ARG);
    const void* ptrs[] = {cu_seqlens, state_pool, init_slot, final_slot, track_chunk_idx, track_state, workspace};
    for (const void* p : ptrs) KDA_REQUIRE(aligned16(p), KDA_ERR_INVALID_ARG);
    DecayMaps maps;
    DecayPrefillArgs a{};
    if (T_tot > 0) {
        const LatentRows rq = as_rows(q), rk = as_rows(k), rv = as_rows(v);
        KDA_REQUIRE(chunk_map(&maps.q, in_dtype, rq, Hk, T_tot, kDecayChunk) &&
                        chunk_map(&maps.k, in_dtype, rk, Hk, T_tot, kDecayChunk) &&
                        chunk_map(&maps.v, in_dtype, rv, H, T_tot, kDecayChunk),
                    KDA_ERR_CUDA);
        a.hq = rq.hs != 0, a.hk = rk.hs != 0, a.hv = rv.hs != 0;
        a.out = as_rows(out);
        a.ho = a.out.hs != 0;
        a.boxes = out_dtype == in_dtype && (a.out.hs != 0 || H == 1) && (a.out.rs > 0 || T_tot == 1) && a.out.hs >= 0;
        if (a.boxes) KDA_REQUIRE(chunk_map(&maps.out, out_dtype, a.out, H, T_tot, 32), KDA_ERR_CUDA);
    }
    a.head_decay = head_decay;
    a.log_decay = log_decay;
    a.cu = cu_seqlens;
    a.init_slot = init_slot;
    a.final_slot = final_slot;
    a.track_idx = track_chunk_idx;
    a.pool = state_pool;
    a.track = track_state;
    a.dev_status = dev_status;
    a.P = P;
    a.N = N;
    a.T = T_tot;
    a.H = H;
    a.group = H / Hk;
    a.M = M;
    a.out_dt = out_dtype;
    a.st = state_type(flags);
    a.scale = scale;
    a.give_up_cta = give_up_cta;
    a.give_up_load = give_up_load;
    auto* f = in_dtype == KDA_BF16 ? decay_prefill_kernel<KDA_BF16> : decay_prefill_kernel<KDA_F16>;
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)DS_SMEM) != cudaSuccess)
        return runtime_failed();
    cudaStream_t s = as_stream(stream);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(N * H));
    cfg.blockDim = dim3(kPreDecayThreads);
    cfg.dynamicSmemBytes = DS_SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    if (workspace && may_cut(T_tot)) {
        KDA_REQUIRE(ws_bytes >= kCutBytes, KDA_ERR_INVALID_ARG);
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return runtime_failed();
        const int64_t most = ((int64_t)T_tot / kDecayChunk + (1 + kUnitChunks) * (int64_t)N) * H;  // places
        // The kernel, which sees the lengths, takes one for each kCutChunks places, or one for each pair where those are short,
        // and leaves the rest.  (Without the second: 16 prompts of 70 tokens, 4 heads 24.7 us for 18.6, 16 of 100, 8 heads 30.3
        // for 26.7.)
        const int64_t pairs = (int64_t)N * H, ctas = std::max((most + kCutChunks - 1) / kCutChunks, pairs);
        cfg.gridDim.x = (unsigned)std::min(ctas, (int64_t)(sms < kDecayCtas ? sms : kDecayCtas));
        a.flags = static_cast<uint32_t*>(workspace);
        a.decays = reinterpret_cast<float*>(a.flags + kDecayCtas);
        a.states = a.decays + kDecayCtas;
        if (cudaMemsetAsync(a.flags, 0, 4 * kDecayCtas, s) != cudaSuccess) return runtime_failed();
        at[0].id = cudaLaunchAttributeCooperative;
        at[0].val.cooperative = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    if (cudaLaunchKernelEx(&cfg, f, maps, a) != cudaSuccess) return runtime_failed();
    return launch_status();
}

}  // namespace
}  // namespace kda

extern "C" kda_status kda_decay_prefill(
    const kda_rows_desc* q, const kda_rows_desc* k, const kda_rows_desc* v,
    kda_dtype in_dtype, const float* head_decay, const float* log_decay, const int32_t* cu_seqlens, int32_t N, int32_t T_tot,
    int32_t H, int32_t Hk, int32_t dk, int32_t dv, float scale, uint32_t flags, void* state_pool, int64_t P,
    const int32_t* init_slot, const int32_t* final_slot, const int32_t* track_chunk_idx, int32_t M, void* track_state,
    const kda_rows_desc* out, kda_dtype out_dtype, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
    return prefill_call(q, k, v, in_dtype, head_decay, log_decay, cu_seqlens, N, T_tot, H, Hk, dk, dv, scale, flags, state_pool, P, init_slot,
                        final_slot, track_chunk_idx, M, track_state, out, out_dtype, workspace, ws_bytes, dev_status, stream, -1, 0);
}

extern "C" kda_status kda_selftest_decay_prefill_give_up(
    const kda_rows_desc* q, const kda_rows_desc* k, const kda_rows_desc* v,
    kda_dtype in_dtype, const float* head_decay, const float* log_decay, const int32_t* cu_seqlens, int32_t N, int32_t T_tot,
    int32_t H, int32_t Hk, int32_t dk, int32_t dv, float scale, uint32_t flags, void* state_pool, int64_t P,
    const int32_t* init_slot, const int32_t* final_slot, const int32_t* track_chunk_idx, int32_t M, void* track_state,
    const kda_rows_desc* out, kda_dtype out_dtype, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream,
    int32_t block, int32_t load) {
    KDA_REQUIRE(block >= 0 && load >= 0, KDA_ERR_INVALID_ARG);
    return prefill_call(q, k, v, in_dtype, head_decay, log_decay, cu_seqlens, N, T_tot, H, Hk, dk, dv, scale, flags, state_pool, P, init_slot,
                        final_slot, track_chunk_idx, M, track_state, out, out_dtype, workspace, ws_bytes, dev_status, stream, block, load);
}
