// latent_decode.cu -- kda_latent_decode: absorbed latent attention over a paged cache.
//
// One latent row (1152 bytes) serves every head as key and, its first 1024 bytes, as value, so a
// request's tokens are read once for up to 64 query rows (positions x heads).  Tokens come T = 64
// or 48 at a time; with Q the query rows [N, 576], C a tile [T, 576] and V its first 512 channels:
//   S   = Q C^T          M = 128 (the N rows repeated), N = T tokens, K = 576
//   P   = 2^(c S - m)    c = scale log2 e, m a running maximum of the row
//   O^T += V^T P^T       4 products M = 128 value channels, N rows, K = T tokens
// O stays transposed in TMEM (lane = value channel): 512 fp32 channels of 128 rows would take all
// 512 columns, transposed they take 4 N, and few query rows waste no tensor-core rows in this
// product.  The tile is used as it lies in shared memory: K-major for S, MN-major for V^T.
// m moves only when a row's maximum exceeds it by 8 (a factor of 256; fp16 has room for it, see log2_base):
// rescaling O is then rare, and exact up to fp32 rounding.
//
// Work: all (row tile, request, token tile) triples in one line, cut into equal ranges, one a CTA
// and SM, so ragged and few long requests load every SM alike.  A CTA walks its range through
// whole requests (written as results) and at most two partial ones (unnormalised O, m and l to the
// workspace, joined by combine_kernel).
//
// Roles: warps 0, 2 and 3 load (TMA boxes of one page's rows, a ring of 128-channel pairs so that a
// part is free for the next tile as soon as its product is done), warp 1 issues MMAs, whichever of
// S(i+1) and O(i) is ready first, warps 4-7 do softmax, rescaling, queries and results.
#include "kda_host.h"
#include "latent_common.cuh"
#include "latent_host.h"
#include "umma.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kMaxTile = 64;                // tokens a tile, at most (DecLayout::T)
constexpr int kDecCtas = 152;               // one a SM
constexpr int kDecThreads = 256;
constexpr uint32_t kDecWait = 1u << 18;     // polls, about a second: loads and MMAs take microseconds

struct DecodeArgs {
    LatentRows ql, qr;
    int32_t R, K;
    const int32_t* q_len;
    int32_t H;
    float c;        // |scale| log2 e
    bool negate;    // scale < 0
    int64_t P;
    int32_t page_size, box;  // box: rows of one TMA box, a divisor of page_size and of the tile
    const int32_t* table;
    int32_t max_pages;
    const int32_t* seq_len;
    void* out;
    int64_t out_rs, out_hs;
    int32_t out_dt;
    float* lse;
    int32_t n_rt;   // row tiles of a request
    // Where split requests lie: (r, row tile, first CTA, last CTA), r = -1 for none.  With at most as many
    // (request, row tile)s as CTAs an entry for each of these, else one for each CTA: for the request
    // whose first part, but not the last, it holds.
    int4* meta;
    bool by_unit;
    float2* ml;     // [2 CTAs][N] (log2_base of m, l)
    float* part;    // [2 CTAs][N][512]
    int32_t* dev_status;
    int32_t give_up_cta, give_up_pair;  // of the self-test: this CTA's loads stop before this column pair
};

// The plan of a CTA with N query rows a tile.  Q is the A operand of S with M = 128: its N rows are
// repeated 128 / N times along M, so that every softmax thread has a row and its share of the tile's
// scores.  Q lies in TMEM (32 columns a 64-channel part) as far as there are columns beside O and S:
// all of it for N <= 32, six parts of nine for N = 64, the rest in shared memory.  An S product then
// reads 2 KiB of shared memory instead of 6 (a product of M = 128, N = 64, K = 16 is bound by that:
// 44 cycles against 32), and the shared memory saved holds a third tile in flight.  With N = 64 three
// tiles fit at 48 tokens each: two and a quarter of 64 did not cover the chain load, S, softmax, O of a
// tile (64 x 7 positions of about 6000 tokens, 32 heads: 310 us with 48, 329 with 64, before later steps).
template <int N>
struct DecLayout {
    static constexpr int T = N == 64 ? 48 : 64;       // tokens a tile
    static constexpr uint32_t COL = T * 128;          // bytes of a 64-channel column of a tile
    static constexpr int REP = 128 / N;               // copies of a row along M
    static constexpr int CW = T / REP;                // scores a thread and tile
    static constexpr int QT = N == 64 ? 6 : 9;        // parts of Q in TMEM
    static constexpr int PAIRS = 12, ROPES = 3;       // rings of column pairs (4 a tile) and rope columns
    static constexpr int NP = N == 64 ? 1 : 2;        // buffers of P
    static constexpr uint32_t QS = 0;                 // parts QT .. 8 of Q, 128 rows
    static constexpr uint32_t PAIR = QS + (9 - QT) * 128 * 128;
    static constexpr uint32_t ROPE = PAIR + PAIRS * 2 * COL;
    static constexpr uint32_t P = ROPE + ROPES * COL;
    static constexpr uint32_t MISC = P + NP * N * 128;
    // two 64-channel columns of all rows, on their way into TMEM: P is free then, and so is QS until its
    // own parts come
    static constexpr uint32_t STAGE = N == 64 ? QS + 2 * 128 * 128 : P;
    static constexpr int B_FULL = 0, B_EMPTY = PAIRS, B_RFULL = 2 * PAIRS, B_REMPTY = B_RFULL + ROPES,
                         B_S = B_REMPTY + ROPES, B_SFREE = B_S + 1, B_P = B_SFREE + 1, B_PV = B_P + 2, B_Q = B_PV + 2,
                         B_DRAIN = B_Q + 1, BARS = B_DRAIN + 1;
    static constexpr uint32_t ROWF = MISC + 8 * 40;      // [N] row factors
    static constexpr uint32_t BAD = ROWF + 4 * N;        // [ROPES] bad boxes of the tile in a rope slot
    static constexpr uint32_t CTRL = BAD + 16;           // tmem address, dead flag, start of the range
    static constexpr uint32_t SCAN = CTRL + 48;          // [2][8] warp sums
    static constexpr uint32_t ROWO = SCAN + 128;         // [N] output offsets of the rows
    static constexpr uint32_t PMAX = ROWO + 8 * N;       // [2][128] partial maxima
    static constexpr uint32_t SMEM = PMAX + 1024;
    static constexpr uint32_t TM_S = 4 * N, TM_Q = TM_S + 64;
    static_assert(4 * ROPES <= PAIRS, "the loads waited for at the end are the last of their slots");
    static_assert(BARS <= 40 && SMEM <= 232448 && TM_Q + 32 * QT <= 512, "shared memory and TMEM plan");
};

// Length and query count of a request as the kernel uses them: an invalid one has none.  One without
// query positions has no length either: nothing of what its table and pages hold is read.
__device__ __forceinline__ int request(const DecodeArgs& a, int r, int& ql, int& err) {
    int len = a.seq_len[r];
    ql = a.q_len ? a.q_len[r] : a.K;
    err = 0;
    if (len < 0 || len > (int64_t)a.max_pages * a.page_size) {
        err = KDA_DEV_BAD_SEQLEN;
        len = 0;
    }
    if (ql < 0 || ql > a.K) {
        err |= KDA_DEV_BAD_ACCEPT;
        ql = 0;
    }
    return ql > 0 ? len : 0;
}
// token tiles of a request; one without tokens takes one (empty) tile, for its zero rows
template <int N>
__device__ __forceinline__ int tiles_of(int len) {
    return len > 0 ? (len + DecLayout<N>::T - 1) / DecLayout<N>::T : 1;
}
// Turning to another request (its queries in, the last one's results out) takes as long as some tiles:
// every request counts so much longer in the line of work that is cut into equal ranges (256 requests of
// about 64 tiles 209 -> 207 us, four of 2048 tiles 110 -> 108.5 us; 64 requests of 7 positions 318 us without,
// 311.5 with 3 tiles, 307 with 6).  Not with few tiles a CTA, where a tile more on one of them would cost more.
constexpr int turn_of(int N, long long tiles, int ctas) { return tiles < 8ll * ctas ? 0 : N == 64 ? 6 : 2; }

// The walk over a CTA's range: next() gives the tiles [j0, j1) of request r, row tile rt.
template <int N>
struct Walk {
    int r, rt, j, turn;
    long long left;
    int j0, j1, n, len, ql, err;
    int cr, crt;
    __device__ __forceinline__ bool next(const DecodeArgs& a) {
        while (left > 0) {
            cr = r;
            crt = rt;
            len = request(a, r, ql, err);
            n = tiles_of<N>(len);
            const int all = n + turn;
            const int end = (long long)(all - j) <= left ? all : j + (int)left;
            j0 = j;
            j1 = min(end, n);
            left -= end - j;
            j = end;
            if (j == all) {
                j = 0;
                if (++r == a.R) {
                    r = 0;
                    ++rt;
                }
            }
            if (j0 < j1) return true;  // else only the turn falls into this range
        }
        return false;
    }
};

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// This thread's CW scores: columns col0 .. of its TMEM lane.  A load's address is the warp's, so with
// CW = 8 (two copies of the rows in a warp) each half of the warp takes its half of 16 columns.
template <int CW>
__device__ __forceinline__ void ld_scores(uint32_t taddr, int col0, int lane, float (&v)[CW]) {
    static_assert(CW == 8 || CW == 16 || CW == 24, "one 16-column load, and one of 8 for 24");
    uint32_t u[16], w[8];
    const uint32_t base = taddr + (CW < 16 ? col0 & ~15 : col0);
    ld16_issue(base, u);
    if constexpr (CW == 24)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "r"(base + 16));
    wait_ld();
#pragma unroll
    for (int i = 0; i < CW; ++i)
        v[i] = __uint_as_float(CW < 16 && lane >= 16 ? u[(8 + i) & 15] : i < 16 ? u[i & 15] : w[i & 7]);
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// kGiveUp: the self-test's form, in which one wait of a loading warp counts as run out.
template <int N, int DT, bool kGiveUp>
__global__ void __launch_bounds__(kDecThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap rmap,
                  const __grid_constant__ DecodeArgs a) {
    using L = DecLayout<N>;
    using E = Elem<DT>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) { return sb + L::MISC + 8 * i; };
    float* rowf = reinterpret_cast<float*>(sm + L::ROWF);
    float* pmax = reinterpret_cast<float*>(sm + L::PMAX);
    volatile int* bad_box = reinterpret_cast<int*>(sm + L::BAD);
    volatile int* ctrl = reinterpret_cast<int*>(sm + L::CTRL);  // 0 tmem, 1 dead, 2 r, 3 rt, 4 j
    int64_t* rowo = reinterpret_cast<int64_t*>(sm + L::ROWO);
    long long* scan = reinterpret_cast<long long*>(sm + L::SCAN);
    const float inf = __int_as_float(0x7f800000);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid < L::BARS) mbar_init(bar(tid), tid == L::B_P || tid == L::B_P + 1 || tid == L::B_Q || tid == L::B_SFREE ? 4 : 1);
    if (tid == 0) {
        ctrl[1] = 0;
        ctrl[2] = -1;
    }
    if (tid == 64) prefetch_map(&map);
    if (tid == 96) prefetch_map(&rmap);
    if (warp == 1) tmem_alloc(sb + L::CTRL, 512);

    // ---- this CTA's range: the tiles of all requests, then the request its start falls into
    auto tiles_at = [&](int r) {
        int ql, err;
        return r < a.R ? (long long)tiles_of<N>(request(a, r, ql, err)) : 0ll;
    };
    auto inclusive = [&](long long x) {  // over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    long long n = tiles_at(tid), more_n = 0;  // of the first requests, one a thread, and of the others
    for (int r = tid + kDecThreads; r < a.R; r += kDecThreads) more_n += tiles_at(r);
    long long x = inclusive(n);
    more_n = inclusive(more_n);
    if (lane == 31) {
        scan[warp] = x;
        scan[8 + warp] = more_n;
    }
    __syncthreads();
    long long S = 0, before = 0, off = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w < warp) off += scan[w];
        before += scan[w];
        S += scan[w] + scan[8 + w];
    }
    const int turn = turn_of(N, S * a.n_rt, gridDim.x);
    S += (long long)turn * a.R;
    const long long T = S * a.n_rt;
    const long long G = T < gridDim.x ? T : gridDim.x;  // CTAs with work
    const bool work = blockIdx.x < G;
    const long long g0 = work ? T * blockIdx.x / G : 0, g1 = work ? T * (blockIdx.x + 1) / G : 0;
    const int rt0 = (int)(g0 / S);
    const long long want = g0 - rt0 * S;
    auto found = [&](int r) {
        const long long lo = off + x - n + (long long)turn * r;
        if (n > 0 && want >= lo && want < lo + n + turn) {
            ctrl[2] = r;
            ctrl[3] = rt0;
            ctrl[4] = (int)(want - lo);
            // the first pages of the range: they are asked for before the CTA is set up
            const int64_t page = min((want - lo) * L::T / a.page_size, (long long)a.max_pages - 1);
            if (page >= 0) prefetch_l2(a.table + (int64_t)r * a.max_pages + page);
        }
    };
    found(tid);
    for (int base = kDecThreads; base < a.R && before + (long long)turn * base <= want; base += kDecThreads) {
        __syncthreads();
        n = tiles_at(base + tid);
        x = inclusive(n);
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        off = before;
        for (int w = 0; w < 8; ++w) {
            if (w < warp) off += scan[w];
            before += scan[w];
        }
        found(base + tid);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = ctrl[0];
    auto range = [&] {
        Walk<N> w;
        w.r = ctrl[2];
        w.rt = ctrl[3];
        w.j = ctrl[4];
        w.turn = turn;
        w.left = w.r < 0 ? 0 : g1 - g0;
        return w;
    };
    Walk<N> w = range();
    bool dead = false;
    // a wait that gives up marks the CTA: every role leaves its loop at its next wait
    auto give_up = [&] {
        dead = true;
        ctrl[1] = 1;
        report(a.dev_status, KDA_DEV_TIMEOUT);
    };
    auto wait = [&](int b, uint32_t parity) {
        if (dead) return;
        if (!mbar_wait(bar(b), parity, kDecWait)) give_up();
    };

    if (warp == 0 || warp == 2 || warp == 3) {
        // ================================================================ loads
        // warp 0: the rope part and, with 64-row boxes, everything (5 boxes a tile: a pair is one box
        // of two 64-channel columns); with smaller boxes (8 pages or fewer a tile, 9 boxes each)
        // warps 2 and 3 take two pairs each, since one warp issues a box in some 100 cycles
        const bool whole_box = a.box == kMaxTile;
        const int part = warp;  // 0: rope (and pairs 0..3), 2: pairs 0, 1, 3: pairs 2, 3
        const int p_lo = part == 3 ? 2 : 0, p_hi = whole_box ? (part == 0 ? 4 : 0) : part == 0 ? 0 : p_lo + 2;
        const uint32_t per = L::T / a.box;
        uint32_t tile = 0, pairs = 0, ropes = 0;  // tiles done; column pairs and rope columns asked for
        while (!dead && w.next(a)) {
            const int32_t* tab = a.table + (int64_t)w.cr * a.max_pages;
            // page of this lane's box in tile j (-1: none) and the box's first row in it
            auto page_of = [&](int j, uint32_t& y) {
                const uint32_t t = (uint32_t)j * L::T + lane * a.box;
                const uint32_t pg = t / (uint32_t)a.page_size;
                y = t - pg * a.page_size;
                return lane < (int)per && t < (uint32_t)w.len ? tab[pg] : INT32_MIN;
            };
            uint32_t ynext = 0;
            int next = page_of(w.j0, ynext);
            for (int j = w.j0; j < w.j1 && !dead; ++j, ++tile) {
                const int page = next;
                const uint32_t y = ynext;
                const bool has = lane < (int)per && (uint32_t)j * L::T + lane * a.box < (uint32_t)w.len;
                if (j + 1 < w.j1) next = page_of(j + 1, ynext);
                const bool ok = has && page >= 0 && page < a.P;
                const uint32_t okm = __ballot_sync(~0u, ok);
                const uint32_t badm = __ballot_sync(~0u, has && !ok);
                const uint32_t bytes = (uint32_t)__popc(okm) * a.box * 128;
                for (int p = p_lo; p < p_hi; ++p) {
                    const uint32_t n = tile * 4 + p, slot = n % L::PAIRS;
                    wait(L::B_EMPTY + slot, (n / L::PAIRS & 1) ^ 1);  // the first pass finds the slots free
                    if (kGiveUp && !dead && (int)blockIdx.x == a.give_up_cta && (int)n == a.give_up_pair) give_up();
                    dead = __any_sync(~0u, dead);
                    if (dead) break;
                    if (lane == 0) mbar_expect_tx(bar(L::B_FULL + slot), 2 * bytes);
                    __syncwarp();
                    if (ok) {
                        const uint32_t dst = sb + L::PAIR + slot * (2 * L::COL) + lane * a.box * 128;
                        tma_load_4d(dst, &map, 0, y, 2 * p, page, bar(L::B_FULL + slot));
                        if (!whole_box)
                            tma_load_4d(dst + L::COL, &map, 0, y, 2 * p + 1, page, bar(L::B_FULL + slot));
                    }
                    ++pairs;
                }
                if (dead) break;
                if (part == 0) {
                    const uint32_t slot = tile % L::ROPES;
                    wait(L::B_REMPTY + slot, (tile / L::ROPES & 1) ^ 1);
                    dead = __any_sync(~0u, dead);
                    if (dead) break;
                    if (lane == 0) {
                        if (badm) report(a.dev_status, KDA_DEV_BAD_SLOT);
                        bad_box[slot] = (int)badm;
                        mbar_expect_tx(bar(L::B_RFULL + slot), bytes);
                    }
                    __syncwarp();
                    if (ok)
                        tma_load_4d(sb + L::ROPE + slot * L::COL + lane * a.box * 128, &rmap, 0, y, 8, page,
                                    bar(L::B_RFULL + slot));
                    ++ropes;
                }
            }
            if (ctrl[1]) dead = true;
            dead = __any_sync(~0u, dead);
        }
        // Nothing may be in flight when the CTA ends: the last loads of this warp have landed, those of a tile
        // that was given up half asked for among them.  Each wait is bounded by itself: one that runs out
        // does not let the others pass.
        auto landed = [&](int b, uint32_t parity) {
            dead = false;
            wait(b, parity);
        };
        const uint32_t per_tile = p_hi - p_lo;
        for (uint32_t k = pairs - min(pairs, L::ROPES * per_tile); k < pairs; ++k) {
            const uint32_t n = k / per_tile * 4 + p_lo + k % per_tile;
            landed(L::B_FULL + n % L::PAIRS, n / L::PAIRS & 1);
        }
        for (uint32_t k = ropes - min(ropes, (uint32_t)L::ROPES); k < ropes; ++k)
            landed(L::B_RFULL + k % L::ROPES, k / L::ROPES & 1);
    } else if (warp == 1) {
        // ================================================================ MMAs
        // the whole warp runs this, one lane issues (umma.cuh, mma_by); votes keep the control uniform
        const uint32_t lead = elect_lane();
        const uint32_t sb4 = sb >> 4;
        const uint32_t tm = __shfl_sync(~0u, tmem, 0);
        const uint32_t ids = idesc_16(DT == KDA_F16, 128, L::T, false, false, a.negate);
        const uint32_t idv = idesc_16(DT == KDA_F16, 128, N, true, false, false);
        Walk<N> ws = w;  // S runs ahead of O, over its own copy of the walk
        bool more_s = __any_sync(~0u, ws.next(a)), more_v = __any_sync(~0u, w.next(a));
        int js = ws.j0, jv = w.j0;
        bool first_s = true, first_v = true;          // of a segment
        uint32_t s_it = 0, v_it = 0;                  // tiles issued
        uint32_t s_slot = 0, s_ph = 0, v_slot = 0, r_slot = 0, r_ph = 0, vr_slot = 0, segs = 0;
        uint32_t idle = 0;
        bool stop = false;
        while (more_v && !stop) {
            bool did = false;
            if (v_it < s_it && __all_sync(~0u, mbar_test(bar(L::B_P + v_it % L::NP), v_it / L::NP & 1))) {
                fence_after();
                const uint32_t p4 = sb4 + L::P / 16 + v_it % L::NP * (N * 128 / 16);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t a4 = sb4 + L::PAIR / 16 + v_slot * (2 * L::COL / 16);
#pragma unroll
                    for (int s = 0; s < L::T / 16; ++s)
                        mma_by(lead, tm + c * N, desc_mn4(a4, L::COL, 1024, s), desc_k4(p4, N, s), idv,
                               s != 0 || !first_v);
                    commit_by(lead, bar(L::B_EMPTY + v_slot));
                    if (++v_slot == L::PAIRS) v_slot = 0;
                }
                // the rope slot goes back with the tile, not with S: the softmax of this tile has
                // read the slot's bad boxes and waited on its barrier by now
                commit_by(lead, bar(L::B_REMPTY + vr_slot));
                if (++vr_slot == L::ROPES) vr_slot = 0;
                commit_by(lead, bar(L::B_PV + v_it % L::NP));
                ++v_it;
                first_v = __any_sync(~0u, ++jv == w.j1);
                if (first_v) {
                    more_v = __any_sync(~0u, w.next(a));
                    jv = w.j0;
                }
                did = true;
            }
            if (more_s) {
                const bool t0 = mbar_test(bar(L::B_RFULL + r_slot), r_ph);  // loaded last
                const bool t1 = mbar_test(bar(L::B_SFREE), (s_it & 1) ^ 1);  // free at first
                const bool t2 = mbar_test(bar(L::B_Q), (segs & 1) ^ !first_s);
                if (__all_sync(~0u, t0 & t1 & t2)) {
                    if (first_s) ++segs;
                    const uint32_t d = tm + L::TM_S;
#pragma unroll
                    for (int c = 0; c < 9; ++c) {
                        uint32_t b4;
                        if (c < 8) {
                            if (c % 2 == 0) {
                                wait(L::B_FULL + s_slot, s_ph);
                                fence_after();
                            }
                            b4 = sb4 + L::PAIR / 16 + s_slot * (2 * L::COL / 16) + (c % 2) * (L::COL / 16);
                        } else {
                            b4 = sb4 + L::ROPE / 16 + r_slot * (L::COL / 16);
                        }
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            if (c < L::QT)
                                mma_ta_by(lead, d, tm + L::TM_Q + 32 * c + 8 * s, desc_k4(b4, L::T, s), ids, c + s != 0);
                            else
                                mma_by(lead, d, desc_k4(sb4 + L::QS / 16 + (c - L::QT) * 1024, 128, s),
                                       desc_k4(b4, L::T, s), ids, 1);
                        }
                        if (c < 8 && c % 2 == 1)
                            if (++s_slot == L::PAIRS) s_slot = 0, s_ph ^= 1;
                    }
                    commit_by(lead, bar(L::B_S));
                    if (++r_slot == L::ROPES) r_slot = 0, r_ph ^= 1;
                    ++s_it;
                    first_s = __any_sync(~0u, ++js == ws.j1);
                    if (first_s) {
                        more_s = __any_sync(~0u, ws.next(a));
                        js = ws.j0;
                    }
                    did = true;
                }
            }
            // polls of some tens of cycles: it gives up after about a second without work.  Nothing else is asked
            // after a product: this warp's instructions between products bound a tile of N = 64 (votes on
            // dead and ctrl each time cost 6 % for 64 x 7 positions).
            if (did) {
                idle = 0;
            } else {
                ++idle;
                stop = __any_sync(~0u, dead || idle > (1u << 23) || ctrl[1]);
            }
        }
        if (stop && lane == 0) {
            ctrl[1] = 1;
            report(a.dev_status, KDA_DEV_TIMEOUT);
        }
        commit_by(lead, bar(L::B_DRAIN));
        dead = false;
        wait(L::B_DRAIN, 0);
    } else if (warp >= 4) {
        // ================================================================ softmax, queries, results
        constexpr int CW = L::CW, NR = N == 64 ? 2 : 1;
        const int q4 = warp - 4, t = tid - 128;
        const uint32_t tq = tmem + ((uint32_t)(q4 * 32) << 16);
        const int row = t % N, col0 = t / N * CW;  // this thread's query row and first score
        uint32_t it = 0, rslot = 0, rph = 0;
        // The queries of a row tile: read from global memory along the rows (16 threads a row's 256
        // bytes), turned in shared memory, 128 channels at a time, and written by the thread that
        // has the row to its TMEM lane; the parts without columns go to shared memory.
        auto load_q = [&](int r, int rt) {
            uint4 v[N / 8][5];
#pragma unroll
            for (int i = 0; i < N / 8; ++i) {
                const int f = rt * N + 8 * i + (t >> 4);
                const int tt = f / a.H, h = f - tt * a.H;
                const int64_t qrow = (int64_t)r * a.K + tt;
                const uint4* ql = reinterpret_cast<const uint4*>(a.ql.base + qrow * a.ql.rs + h * a.ql.hs) + (t & 15);
                const uint4* qr = reinterpret_cast<const uint4*>(a.qr.base + qrow * a.qr.rs + h * a.qr.hs) + (t & 15);
#pragma unroll
                for (int g = 0; g < 5; ++g) {
                    v[i][g] = make_uint4(0, 0, 0, 0);
                    if (f < a.K * a.H) {
                        if (g < 4) v[i][g] = __ldg(ql + 16 * g);
                        else if ((t & 15) < 8) v[i][g] = __ldg(qr);
                    }
                }
            }
            // the last product that reads P (and so every earlier one) is done
            if (it > 0) wait(L::B_PV + (it - 1) % L::NP, (it - 1) / L::NP & 1);
#pragma unroll
            for (int g = 0; g < 5; ++g) {
                const uint32_t stage = sb + (g < 4 ? L::STAGE : L::P);  // the last is one column: P has room for it
                if (g) bar_named(1, 128);
#pragma unroll
                for (int i = 0; i < N / 8; ++i) {
                    if (g == 4 && (t & 15) >= 8) continue;
                    const int rr = 8 * i + (t >> 4);
                    sts16(stage + ((t >> 3) & 1) * (N * 128) + rr * 128 + (((t ^ rr) & 7) << 4), v[i][g]);
                }
                bar_named(1, 128);
#pragma unroll
                for (int c = 2 * g; c < 2 * g + 2 && c < 9; ++c) {
                    uint32_t u[2][16];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const uint4 y = lds16(stage + (c & 1) * (N * 128) + row * 128 + (((x ^ row) & 7) << 4));
                        const int o = 4 * (x & 3);
                        u[x >> 2][o] = y.x, u[x >> 2][o + 1] = y.y, u[x >> 2][o + 2] = y.z, u[x >> 2][o + 3] = y.w;
                        if (c >= L::QT) sts16(sb + L::QS + chunk_k(t, (c - L::QT) * 64 + 8 * x, 128), y);
                    }
                    if (c < L::QT) {
                        st16u(tq + L::TM_Q + 32 * c, u[0]);
                        st16u(tq + L::TM_Q + 32 * c + 16, u[1]);
                    }
                }
            }
            wait_st();
            if (L::QT < 9) fence_async_smem();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::B_Q));
        };
        if (t == 0 && !a.by_unit) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
        bool more = w.next(a), quit = false;  // quit: agreed by the four warps, so that barriers stay matched
        if (more) load_q(w.cr, w.crt);
        while (more && !quit) {
            const Walk<N> g = w;  // this segment
            if (t == 0 && g.j0 == 0 && g.crt == 0 && g.err) report(a.dev_status, g.err);
            // the running maximum of this thread's row and, for N = 64, of the row its warp does not
            // hold: every warp then knows by itself whether any row moves its maximum
            float m[NR];
#pragma unroll
            for (int q = 0; q < NR; ++q) m[q] = -inf;
            WeightSum sum;  // over this thread's columns
            int last = -1;  // last token this thread's row sees
            const int f = g.crt * N + row;
            if (f < a.K * a.H) {
                const int tt = f / a.H;
                if (tt < g.ql) last = g.len - g.ql + tt;
            }
            for (int j = g.j0; j < g.j1; ++j, ++it) {
                wait(L::B_S, it & 1);
                wait(L::B_RFULL + rslot, rph);
                fence_after();
                if (j == max(g.j0, g.j1 - 3)) {
                    // the next segment's query rows into L2: behind the loads of the ring, a read from
                    // HBM takes some microseconds, and S waits for it
                    Walk<N> nx = w;
                    if (nx.next(a)) {
                        const int rr = t % N, ff = nx.crt * N + rr, tt = ff / a.H, h = ff - tt * a.H;
                        if (ff < a.K * a.H) {
                            const int64_t qrow = (int64_t)nx.cr * a.K + tt;
                            for (int x = t / N; x < 9; x += L::REP)
                                prefetch_l2(x < 8 ? a.ql.base + qrow * a.ql.rs + h * a.ql.hs + x * 64
                                                  : a.qr.base + qrow * a.qr.rs + h * a.qr.hs);
                        }
                    }
                }
                const int t0 = j * L::T;
                const uint32_t bad = (uint32_t)bad_box[rslot];
                if (++rslot == L::ROPES) rslot = 0, rph ^= 1;
                const int valid = g.len - t0;  // tokens of this tile (may exceed it)
                float s[CW];
                ld_scores(tq + L::TM_S, col0, lane, s);
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_SFREE));
                if (bad) {
#pragma unroll
                    for (int i = 0; i < CW; ++i)
                        if ((bad >> ((col0 + i) / a.box)) & 1) s[i] = -inf;
                }
                const int lim = last - t0 - col0;  // columns 0 .. lim of this thread are seen
                if (lim < CW - 1) {
#pragma unroll
                    for (int i = 0; i < CW; ++i)
                        if (i > lim) s[i] = -inf;
                }
                float mx = s[0];
#pragma unroll
                for (int i = 1; i < CW; ++i) mx = fmaxf(mx, s[i]);
                float* pm = pmax + (it & 1) * 128;
                pm[t] = mx;
                quit = bar_named_or(1, 128, dead || ctrl[1]);
                if (quit) break;
                bool need = false;
                float f_old = 1.f;
#pragma unroll
                for (int q = 0; q < NR; ++q) {
                    const int r = q ? row ^ 32 : row;
                    float mt = pm[r];
#pragma unroll
                    for (int k = 1; k < L::REP; ++k) mt = fmaxf(mt, pm[r + k * N]);
                    if (j == g.j0) {
                        m[q] = mt;
                    } else if (mt > m[q] && (m[q] == -inf || (mt - m[q]) * a.c > 8.f)) {
                        const float x = ex2((m[q] - mt) * a.c);
                        if (q == 0) f_old = x;
                        m[q] = mt;
                        need = true;
                    }
                }
                const float mc = m[0] == -inf ? 0.f : log2_base<DT>(m[0], a.c);
                float ls[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < CW; ++i) {
                    s[i] = ex2(fmaf(s[i], a.c, -mc));
                    ls[i & 1] += s[i];
                }
                sum.scale(f_old);
                sum.add(ls[0] + ls[1]);
                if (__any_sync(~0u, need)) {  // the same in all four warps
                    if (t < N) rowf[row] = f_old;
                    bar_named(1, 128);
                    wait(L::B_PV + (it - 1) % L::NP, (it - 1) / L::NP & 1);
                    fence_after();
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int n0 = 0; n0 < N; n0 += 16) {
                            float o[16];
                            ld16(tq + c * N + n0, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= rowf[n0 + i];
                            st16f(tq + c * N + n0, o);
                        }
                    wait_st();
                    bar_named(1, 128);  // rowf has been read
                }
                if (it >= L::NP) wait(L::B_PV + it % L::NP, (it - L::NP) / L::NP & 1);  // this P buffer's last product
#pragma unroll
                for (int i = 0; i < CW; i += 8)
                    sts16(sb + L::P + it % L::NP * (N * 128) + chunk_k(row, col0 + i, N),
                          make_uint4(E::put2(s[i], s[i + 1]), E::put2(s[i + 2], s[i + 3]),
                                     E::put2(s[i + 4], s[i + 5]), E::put2(s[i + 6], s[i + 7])));
                if (valid < L::T || bad) {
                    // tokens that are not there: their weight is zero, and so has to be the value
                    // (what lies in the buffer, or past the end of a page, may be anything)
                    // a thread clears one 16-byte word (of 64) of every other token
                    const int x = t & 63;
                    const uint32_t at = sb + L::PAIR + (it * 4 + (x >> 4)) % L::PAIRS * (2 * L::COL) +
                                        ((x >> 3) & 1) * L::COL + (x & 7) * 16;
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    for (int k = max(valid, 0) + (t >> 6); k < L::T; k += 2) sts16(at + k * 128, zero);
                    if (bad)
                        for (int k = t >> 6; k < L::T; k += 2)
                            if ((bad >> (k / a.box)) & 1) sts16(at + k * 128, zero);
                }
                fence_async_smem();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_P + it % L::NP));
            }
            if (quit) break;
            // the next segment's queries: every S of this one has been read
            more = w.next(a);
            if (more) load_q(w.cr, w.crt);
            // results of this segment
            const bool whole = g.j0 == 0 && g.j1 == g.n;
            const int slot = 2 * (int)blockIdx.x + (g.j0 == 0);
            const int rows = min(N, a.K * a.H - g.crt * N);
            float l = sum.total();
            pmax[(it & 1) * 128 + t] = l;  // the buffer that the last tile did not use
            bar_named(1, 128);
            if (t < N) {
#pragma unroll
                for (int k = 1; k < L::REP; ++k) l += pmax[(it & 1) * 128 + row + k * N];
                rowf[row] = l == 0.f ? 0.f : 1.f / l;
                rowo[row] = ((int64_t)g.cr * a.K + f / a.H) * a.out_rs + (f % a.H) * a.out_hs;
                const float m2 = m[0] == -inf ? -inf : log2_base<DT>(m[0], a.c);
                if (!whole) {
                    a.ml[(int64_t)slot * N + row] = make_float2(m2, l);
                } else if (a.lse != nullptr && row < rows) {
                    const int tt = f / a.H, h = f - tt * a.H;
                    a.lse[((int64_t)g.cr * a.K + tt) * a.H + h] = l == 0.f ? -inf : (m2 + log2f(l)) * 0.69314718055994531f;
                }
            }
            if (t == 0 && !whole && g.j0 == 0) {
                // the last CTA with a part of this request
                const long long end = g1 + (g.n - g.j1);  // this part ends the range; of the request's tiles
                long long last_cta = (end - 1) * G / T;
                while (T * (last_cta + 1) / G < end) ++last_cta;
                while (T * last_cta / G >= end) --last_cta;
                a.meta[a.by_unit ? g.crt * a.R + g.cr : blockIdx.x] = make_int4(g.cr, g.crt, blockIdx.x, (int)last_cta);
            } else if (t == 0 && whole && a.by_unit) {
                a.meta[g.crt * a.R + g.cr] = make_int4(-1, 0, 0, 0);
            }
            bar_named(1, 128);
            wait(L::B_PV + (it - 1) % L::NP, (it - 1) / L::NP & 1);
            fence_after();
            // channel c * 128 + t of every row; put is chosen once
            auto emit = [&](auto put) {
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int n0 = 0; n0 < N; n0 += 16) {
                        if (n0 >= rows) break;
                        float o[16], fac[16];
                        int64_t off[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) fac[i] = rowf[n0 + i], off[i] = rowo[n0 + i];
                        ld16(tq + c * N + n0, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (n0 + i < rows) put(n0 + i, off[i], c * 128 + t, o[i], fac[i]);
                    }
            };
            if (!whole) {
                float* part = a.part + (int64_t)slot * N * kLatent;
                emit([&](int rr, int64_t, int ch, float x, float) { part[rr * kLatent + ch] = x; });
            } else if (a.out_dt == KDA_BF16) {
                auto* o = static_cast<__nv_bfloat16*>(a.out);
                emit([&](int, int64_t at, int ch, float x, float f) { o[at + ch] = __float2bfloat16_rn(x * f); });
            } else if (a.out_dt == KDA_F16) {
                auto* o = static_cast<__half*>(a.out);
                emit([&](int, int64_t at, int ch, float x, float f) { o[at + ch] = __float2half_rn(x * f); });
            } else {
                auto* o = static_cast<float*>(a.out);
                emit([&](int, int64_t at, int ch, float x, float f) { o[at + ch] = x * f; });
            }
            fence_before();
            // rowf read by all before the next segment writes it.  A row without keys gets its zeros here and
            // not from its factor: beside a NaN or infinity that other rows see, its sums are NaN (a choice
            // for each element above cost 1 to 2 % of the call).
            // Rows whose last product was given up get NaN.
            if (bar_named_or(1, 128, whole && (dead || (t < rows && rowf[t & (N - 1)] == 0.f)))) {
                const bool gone = bar_named_or(1, 128, dead);
                for (int n = 0; n < rows; ++n) {
                    if (!gone && rowf[n] != 0.f) continue;
                    for (int c = t; c < kLatent; c += 128)
                        if (a.out_dt == KDA_F32)
                            static_cast<uint32_t*>(a.out)[rowo[n] + c] = gone ? 0x7fffffffu : 0u;
                        else
                            static_cast<uint16_t*>(a.out)[rowo[n] + c] = gone ? 0x7fff : 0;
                }
                bar_named(1, 128);
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    // A wait that ran out leaves parts unwritten, and the workspace may hold an earlier call's in their place:
    // this CTA's parts turn what they are joined with to NaN, and a request that starts here is not joined.
    if (ctrl[1]) {
        const float nan = __int_as_float(0x7fffffff);
        if (tid < 2 * N) a.ml[(int64_t)blockIdx.x * 2 * N + tid] = make_float2(nan, nan);
        if (tid == 0) {
            if (!a.by_unit) a.meta[blockIdx.x].x = -1;
            else
                for (Walk<N> u = range(); u.next(a);)
                    if (u.j0 == 0) a.meta[u.crt * a.R + u.cr].x = -1;
        }
    }
}

// Joins the parts of a request that several CTAs hold: o = sum_i 2^{m_i - m} O_i / sum_i 2^{m_i - m} l_i.
// Entry blockIdx.x of meta; 128 threads a row, 4 channels a thread.
//   few requests over many CTAs (kSplit): block y has row y, and its four groups of 128 threads a
//     quarter of the parts each;
//   else: one group, rows 4y .. 4y + 3 side by side in each thread (a row a group took four waves of
//     blocks, each as long as its chain of dependent loads: 17 us against 6 for 256 units of 64 rows).
struct Split {
    int r, rt, g, parts;
};
__device__ __forceinline__ Split split_at(const DecodeArgs& a, int e) {
    const int4 me = a.meta[e];
    // an entry of no request, or (after a wait ran out) none that this call wrote
    const bool ok = me.x >= 0 && me.x < a.R && me.y >= 0 && me.y < a.n_rt && me.z >= 0 && me.w >= me.z && me.w < kDecCtas;
    return {me.x, me.y, me.z, ok ? me.w - me.z + 1 : 0};
}
// place of part i (CTA g + i's): the first part in its CTA's second place, the others in the first
template <int N>
__device__ __forceinline__ int64_t part_at(int g, int i, int row) { return (int64_t)(2 * (g + i) + (i == 0)) * N + row; }

// The factors of a row's parts, by one warp: fac[i] = 2^{m_i - m}; returns (m, l) in every lane.
template <int N>
__device__ __forceinline__ float2 part_factors(const DecodeArgs& a, int g, int parts, int row, float* fac, int lane) {
    constexpr int n = (kDecCtas + 31) / 32;
    const float inf = __int_as_float(0x7f800000);
    float2 ml[n];
    float m = -inf, l = 0.f;
#pragma unroll
    for (int k = 0; k < n; ++k) {
        const int i = lane + 32 * k;
        ml[k] = i < parts ? a.ml[part_at<N>(g, i, row)] : make_float2(-inf, 0.f);
        m = fmaxf(m, ml[k].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    const float mr = m == -inf ? 0.f : m;
#pragma unroll
    for (int k = 0; k < n; ++k) {
        const float f = ex2(ml[k].x - mr);
        l = fmaf(f, ml[k].y, l);
        if (lane + 32 * k < parts) fac[lane + 32 * k] = f;
    }
    return make_float2(mr, warp_sum(l));
}
__device__ __forceinline__ void fma4(float4& o, float f, float4 x) {
    o.x = fmaf(f, x.x, o.x);
    o.y = fmaf(f, x.y, o.y);
    o.z = fmaf(f, x.z, o.z);
    o.w = fmaf(f, x.w, o.w);
}
__device__ __forceinline__ void put_row(const DecodeArgs& a, const Split& u, int f, float2 ml, float4 o, int t) {
    const float il = ml.y == 0.f ? 0.f : 1.f / ml.y;
    const int tt = f / a.H, h = f - tt * a.H;
    const int64_t orow = (int64_t)u.r * a.K + tt;
    if (il == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);  // no key, as in decode_kernel
    store4_as(a.out, orow * a.out_rs + h * a.out_hs + 4 * t, make_float4(o.x * il, o.y * il, o.z * il, o.w * il), a.out_dt);
    if (t == 0 && a.lse != nullptr)
        a.lse[orow * a.H + h] = ml.y == 0.f ? -__int_as_float(0x7f800000) : (ml.x + log2f(ml.y)) * 0.69314718055994531f;
}

template <int N, bool kSplit>
__global__ void __launch_bounds__(kSplit ? 512 : 128) combine_kernel(const __grid_constant__ DecodeArgs a) {
    __shared__ float fac[4][kDecCtas];
    __shared__ float2 sml[4];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Split u = split_at(a, blockIdx.x);
    if (u.parts == 0) return;
    const int t = threadIdx.x & 127, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* part = a.part + 4 * t;
    const int rows = a.K * a.H - u.rt * N;  // of this row tile, if less than N
    if constexpr (kSplit) {
        __shared__ float4 acc[3][128];
        const int row = blockIdx.y, sub = threadIdx.x >> 7;
        if (row >= rows) return;
        if (warp == 0) {
            const float2 ml = part_factors<N>(a, u.g, u.parts, row, fac[0], lane);
            if (lane == 0) sml[0] = ml;
        }
        __syncthreads();
        float4 o = zero;
#pragma unroll 10
        for (int i = sub; i < u.parts; i += 4)
            fma4(o, fac[0][i], *reinterpret_cast<const float4*>(part + part_at<N>(u.g, i, row) * kLatent));
        if (sub > 0) acc[sub - 1][t] = o;
        __syncthreads();
        if (sub > 0) return;
#pragma unroll
        for (int k = 0; k < 3; ++k) fma4(o, 1.f, acc[k][t]);
        put_row(a, u, u.rt * N + row, sml[0], o, t);
    } else {
        const int row0 = blockIdx.y * 4;
        if (row0 >= rows) return;
        float4 x[2][4], o[4] = {zero, zero, zero, zero};
        // the first two parts are asked for ahead of the factors (a split request has at least two)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[i][k] = i < u.parts ? *reinterpret_cast<const float4*>(part + part_at<N>(u.g, i, row0 + k) * kLatent) : zero;
        const float2 ml = part_factors<N>(a, u.g, u.parts, row0 + warp, fac[warp], lane);
        if (lane == 0) sml[warp] = ml;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i < u.parts) fma4(o[k], fac[k][i], x[i][k]);
#pragma unroll 2
        for (int i = 2; i < u.parts; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                fma4(o[k], fac[k][i], *reinterpret_cast<const float4*>(part + part_at<N>(u.g, i, row0 + k) * kLatent));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (row0 + k < rows) put_row(a, u, u.rt * N + row0 + k, sml[k], o[k], t);
    }
}

int tile_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }

template <int N, int DT, bool kGiveUp = false>
kda_status launch(const CUtensorMap (&map)[2], const DecodeArgs& a, int64_t max_tiles, cudaStream_t s) {
    using L = DecLayout<N>;
    auto* f = decode_kernel<N, DT, kGiveUp>;
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::SMEM) != cudaSuccess)
        return runtime_failed();
    // every (row tile, request) has at least one tile and at most max_tiles
    const int64_t most = (int64_t)a.n_rt * a.R * max_tiles;
    const unsigned grid = (unsigned)(most < kDecCtas ? most : kDecCtas);
    f<<<grid, kDecThreads, L::SMEM, s>>>(map[0], map[1], a);
    if (max_tiles <= 1) return launch_status();  // one tile a request: nothing is split
    // few requests: many parts each (one request of 38 CTAs: 10 us a row a group, 4 us split)
    const int64_t units = (int64_t)a.n_rt * a.R;
    const bool split = units * 4 <= grid;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.by_unit ? (unsigned)units : grid, split ? N : N / 4);
    cfg.blockDim = dim3(split ? 512 : 128);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, split ? combine_kernel<N, true> : combine_kernel<N, false>, a) != cudaSuccess)
        return runtime_failed();
    return launch_status();
}

template <int DT>
kda_status launch_n(const CUtensorMap (&map)[2], const DecodeArgs& a, int64_t max_tiles, cudaStream_t s) {
    const int n = tile_rows((int64_t)a.K * a.H);
    if (n == 16) return launch<16, DT>(map, a, max_tiles, s);
    if (n == 32) return launch<32, DT>(map, a, max_tiles, s);
    return launch<64, DT>(map, a, max_tiles, s);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_latent_decode_workspace_size(int32_t R, int32_t K, int32_t H) {
    if (R < 0 || K < 0 || H < 0) return 16;
    const size_t n = (size_t)tile_rows((int64_t)K * H);
    return align16(kDecCtas * sizeof(int4)) + 2 * kDecCtas * n * (sizeof(float2) + kLatent * sizeof(float));
}

namespace kda {
namespace {

// Both entry points; give_up_cta < 0 for the call itself.
kda_status decode_call(const kda_rows_desc* q_latent, const kda_rows_desc* q_rope, kda_dtype in_dtype, int32_t R, int32_t K,
                       const int32_t* q_len, int32_t H, int32_t d_latent, int32_t d_rope, float scale, const void* cache,
                       int64_t P, int32_t page_size, int64_t page_stride, const int32_t* block_table, int32_t max_pages,
                       const int32_t* seq_len, const kda_rows_desc* out, kda_dtype out_dtype, float* lse, void* workspace,
                       size_t ws_bytes, int32_t* dev_status, void* stream, int32_t give_up_cta, int32_t give_up_pair) {
    KDA_REQUIRE(R >= 0 && K >= 0 && H > 0 && P >= 0 && page_size > 0 && max_pages >= 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(d_latent == kLatent && d_rope == kRope && K <= 16, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((in_dtype == KDA_BF16 || in_dtype == KDA_F16) && any_dtype_ok(out_dtype), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(page_size % 8 == 0 && (int64_t)R * K * H < (1ll << 31), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((int64_t)max_pages * page_size < (1ll << 31) - kMaxTile && P < (1ll << 31), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE(page_stride % 8 == 0 && page_stride >= (int64_t)page_size * kLatentRow, KDA_ERR_INVALID_ARG);
    if (R == 0 || K == 0) return KDA_OK;
    KDA_REQUIRE(isfinite(scale), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(rows_ok(q_latent) && rows_ok(q_rope) && rows_ok(out), KDA_ERR_INVALID_ARG);
    const void* ptrs[] = {seq_len, workspace};
    for (const void* p : ptrs) KDA_REQUIRE(p != nullptr && aligned16(p), KDA_ERR_INVALID_ARG);
    // an empty cache or table is never read: it may have no address
    KDA_REQUIRE(P == 0 || cache != nullptr, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(max_pages == 0 || block_table != nullptr, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(aligned16(cache) && aligned16(block_table), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(aligned16(q_len) && aligned16(lse) && aligned16(dev_status), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(ws_bytes >= kda_latent_decode_workspace_size(R, K, H), KDA_ERR_INVALID_ARG);
    const int n = tile_rows((int64_t)K * H);
    const int box = lowbit_box(page_size, n == 64 ? 16 : kMaxTile);  // divides the tile as well (48 or 64 tokens)
    const void* base = P > 0 ? cache : q_latent->base;  // a map wants an address, though no page is loaded
    CUtensorMap map[2];
    // the cache as (channel of 64, row, 64-channel column, page): one box is `box` rows of one page
    // and one column (a 128-byte swizzle row), or with a whole tile of rows a pair of columns
    const cuuint64_t dims[4] = {64, (cuuint64_t)page_size, 9, (cuuint64_t)(P > 0 ? P : 1)};
    const cuuint64_t strides[3] = {kLatentRow * 2, 128, (cuuint64_t)page_stride * 2};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)box, box == kMaxTile ? 2u : 1u, 1};
    const cuuint32_t rope_boxes[4] = {64, (cuuint32_t)box, 1, 1};
    KDA_REQUIRE(encode_16bit(&map[0], in_dtype, 4, base, dims, strides, boxes), KDA_ERR_CUDA);
    KDA_REQUIRE(encode_16bit(&map[1], in_dtype, 4, base, dims, strides, rope_boxes), KDA_ERR_CUDA);
    DecodeArgs a{as_rows(q_latent), as_rows(q_rope), R, K, q_len, H, log2_scale(scale), scale < 0.f, P, page_size, box,
                 block_table, max_pages, seq_len, const_cast<void*>(out->base), out->row_stride, out->head_stride,
                 out_dtype, lse, (int32_t)(((int64_t)K * H + n - 1) / n), nullptr, false, nullptr, nullptr, dev_status,
                 give_up_cta, give_up_pair};
    a.by_unit = (int64_t)a.n_rt * R <= kDecCtas;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.meta = reinterpret_cast<int4*>(ws);
    ws += align16(kDecCtas * sizeof(int4));
    a.part = reinterpret_cast<float*>(ws);
    ws += (size_t)2 * kDecCtas * n * kLatent * sizeof(float);
    a.ml = reinterpret_cast<float2*>(ws);
    const int tile = n == 64 ? DecLayout<64>::T : DecLayout<32>::T;
    const int64_t max_tiles = ((int64_t)max_pages * page_size + tile - 1) / tile;
    cudaStream_t s = as_stream(stream);
    if (give_up_cta >= 0) return launch<16, KDA_BF16, true>(map, a, max_tiles > 0 ? max_tiles : 1, s);
    if (in_dtype == KDA_BF16) return launch_n<KDA_BF16>(map, a, max_tiles > 0 ? max_tiles : 1, s);
    return launch_n<KDA_F16>(map, a, max_tiles > 0 ? max_tiles : 1, s);
}

}  // namespace
}  // namespace kda

extern "C" kda_status kda_latent_decode(const kda_rows_desc* q_latent, const kda_rows_desc* q_rope,
                                        kda_dtype in_dtype, int32_t R, int32_t K, const int32_t* q_len,
                                        int32_t H, int32_t d_latent, int32_t d_rope, float scale,
                                        const void* cache, int64_t P, int32_t page_size,
                                        int64_t page_stride, const int32_t* block_table,
                                        int32_t max_pages, const int32_t* seq_len,
                                        const kda_rows_desc* out, kda_dtype out_dtype, float* lse,
                                        void* workspace, size_t ws_bytes, int32_t* dev_status,
                                        void* stream) {
    return decode_call(q_latent, q_rope, in_dtype, R, K, q_len, H, d_latent, d_rope, scale, cache, P, page_size, page_stride,
                       block_table, max_pages, seq_len, out, out_dtype, lse, workspace, ws_bytes, dev_status, stream, -1, 0);
}

extern "C" kda_status kda_selftest_latent_decode_give_up(
    const kda_rows_desc* q_latent, const kda_rows_desc* q_rope, kda_dtype in_dtype, int32_t R, int32_t K, const int32_t* q_len,
    int32_t H, int32_t d_latent, int32_t d_rope, float scale, const void* cache, int64_t P, int32_t page_size,
    int64_t page_stride, const int32_t* block_table, int32_t max_pages, const int32_t* seq_len, const kda_rows_desc* out,
    kda_dtype out_dtype, float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream, int32_t block,
    int32_t load) {
    KDA_REQUIRE(block >= 0 && load >= 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(in_dtype == KDA_BF16 && (int64_t)K * H <= 16, KDA_ERR_UNSUPPORTED);
    return decode_call(q_latent, q_rope, in_dtype, R, K, q_len, H, d_latent, d_rope, scale, cache, P, page_size, page_stride,
                       block_table, max_pages, seq_len, out, out_dtype, lse, workspace, ws_bytes, dev_status, stream, block,
                       load);
}
