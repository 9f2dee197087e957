// latent_prefill.cu -- kda_latent_prefill: expanded latent attention of packed sequences.
//
// A pair of CTAs (a cluster of two SMs, one MMA over both) takes 512 query rows of one (sequence,
// head) as two tiles of 256, 128 rows a CTA, and walks the keys 128 at a time.  Per tile of keys and
// tile of queries
//   S = Q K^T       M = 256, N = 128, K = 192 (128 nope, 64 rope: the rope key is loaded from its one
//                   row a token, so it is not repeated per head anywhere)
//   P = 2^(c S - m) c = scale log2 e, one thread a query row; P goes back to TMEM over S, rounded
//                   to the input type, as the A operand of
//   O += P V        M = 256, N = 128, K = 128; V as it lies in shared memory (MN-major)
// Each CTA loads half of K's rows and half of V's channels.  That halves the shared memory a tile
// takes (three tiles in flight beside the 96 KiB of queries; alone a CTA has room for one and a half,
// and its products wait for their keys) and the operand bytes an MMA reads.
// The two query tiles take turns: while the tensor cores work on one, the four warps of the other do
// its exponentials.  m moves only when a row's maximum exceeds it by 8 (a factor of 256; fp16 has room
// for it, see log2_base), so that O is rarely rescaled.
//
// Roles: warps 0-3 and 4-7 softmax of query tile 0 and 1 (and its results), warp 8 loads by TMA (the
// queries, rings of K and V tiles), warp 9 of the first CTA issues the MMAs of both.  Barriers that the
// MMAs wait on lie in the first CTA and take both CTAs' arrivals; completed MMAs arrive in both.
//
// Blocks of rows follow one another without the pair leaving its SMs: the loading warp asks the launch
// hardware for the next block (cluster launch control) under the last tiles of one, so that a block's first
// loads and products run under the last block's results (5 us of about 50 a block otherwise).  Long blocks
// first: see the order of the sequences below, and a sequence's last queries, which have the most keys,
// before its first.
#include "kda_host.h"
#include "latent_common.cuh"
#include "latent_host.h"
#include "umma.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kQTile = 256, kQBlock = 2 * kQTile, kKTile = 128;
constexpr int kRows = 128;               // query rows of a tile in one CTA
constexpr int kPreThreads = 320;
constexpr uint32_t kPreWait = 1u << 18;  // polls, about a second: loads and MMAs take microseconds
constexpr uint32_t kQPart = 128 * 128;   // 128 rows of 64 16-bit channels
constexpr uint32_t kKPart = 64 * 128;    // 64 rows
constexpr int kStages = 3;
constexpr int kAskTiles = 2;             // a block's loads left when the next block is asked for
constexpr int kSorted = 256;             // up to so many sequences are taken by falling length
constexpr uint32_t kKBytes = 3 * kKPart, kVBytes = 128 * 128;  // a CTA's half of a tile

struct PrefillArgs {
    const int32_t* cu_q;
    const int32_t* cu_k;
    int32_t N, Tq, Tk, H;
    int32_t hq, hk, hv;  // 1, or 0 where the heads share a row (head stride 0)
    float c;             // |scale| log2 e
    bool negate;         // scale < 0
    bool full;
    void* out;
    int64_t out_rs, out_hs;
    int32_t out_dt;
    float* lse;
    int32_t* dev_status;
    int32_t give_up_cta, give_up_tile;  // of the self-test: this CTA's loads stop before this tile of V
};

struct PreMaps {
    CUtensorMap q, k, kr, v;
};

// shared memory: Q (2 x 3 parts), the rings, barriers
constexpr uint32_t PS_K = 6 * kQPart, PS_V = PS_K + kStages * kKBytes, PS_BAR = PS_V + kStages * kVBytes;
constexpr int PB_Q = 0, PB_K = 2, PB_V = PB_K + kStages, PB_NEXT = PB_V + kStages, PB_KFREE = PB_NEXT + 1,
              PB_VFREE = PB_KFREE + kStages, PB_S = PB_VFREE + kStages, PB_P = PB_S + 2, PB_P2 = PB_P + 2,
              PB_O = PB_P2 + 2, PB_QFREE = PB_O + 2, PB_EDGE = PB_QFREE + 2, PB_CLC = PB_EDGE + 1, PB_INFO = PB_CLC + 1,
              PB_IFREE = PB_INFO + 2, PB_DRAIN = PB_IFREE + 2, PB_NEVER = PB_DRAIN + 1, PB_BARS = PB_NEVER + 1;
constexpr uint32_t PS_CTRL = PS_BAR + 8 * 40, PS_SCAN = PS_CTRL + 32, PS_CLC = PS_SCAN + 64, PS_INFO = PS_CLC + 16,
                   PS_ORDER = PS_INFO + 2 * 32, PS_START = PS_ORDER + 4 * kSorted, PS_LEN = PS_START + 4 * (kSorted + 1),
                   PS_SUM = (PS_LEN + 4 * kSorted + 7) & ~7u, PS_SMEM = PS_SUM + 8 * 256;
static_assert(PB_BARS <= 40 && PS_CLC % 16 == 0 && PS_SMEM <= 232448, "shared memory plan");
// TMEM: S of the two query tiles, then O
constexpr uint32_t PT_S = 0, PT_O = 256;

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

// Eight results from o[e] as one 16-byte word.
template <int DT>
__device__ __forceinline__ uint4 pack16(const float (&o)[32], int e) {
    return make_uint4(Elem<DT>::put2(o[e], o[e + 1]), Elem<DT>::put2(o[e + 2], o[e + 3]),
                      Elem<DT>::put2(o[e + 4], o[e + 5]), Elem<DT>::put2(o[e + 6], o[e + 7]));
}

// kGiveUp: the self-test's form, in which one wait of a loading warp counts as run out.
template <int DT, bool kGiveUp>
__global__ void __launch_bounds__(kPreThreads, 1)
    prefill_kernel(const __grid_constant__ PreMaps maps, const __grid_constant__ PrefillArgs a) {
    using E = Elem<DT>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* ctrl = reinterpret_cast<int*>(sm + PS_CTRL);  // 0 tmem, 1 sequence, 2 its block, 3 and 4 where its scan stood, 5 NaN if a wait ran out
    volatile int* info = reinterpret_cast<int*>(sm + PS_INFO);  // two blocks' (head, sequence, first row); sequence -1: no more
    int* scan = reinterpret_cast<int*>(sm + PS_SCAN);
    auto bar = [&](int i) { return sb + PS_BAR + 8 * i; };
    const float inf = __int_as_float(0x7f800000);

    if (tid == 32) prefetch_map(&maps.q);
    if (tid == 64) prefetch_map(&maps.k);
    if (tid == 96) prefetch_map(&maps.kr);
    if (tid == 128) prefetch_map(&maps.v);

    // ---- which block of 512 rows
    const uint32_t rank = blockIdx.x & 1;  // in the cluster
    const int y = (blockIdx.x >> 1) / a.H;
    auto blocks_of = [&](int n, bool& bad) {
        const int q0 = a.cu_q[n], q1 = a.cu_q[n + 1], k0 = a.cu_k[n], k1 = a.cu_k[n + 1];
        bad = q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk;
        return bad ? 0 : (q1 - q0 + kQBlock - 1) / kQBlock;
    };
    // Blocks are taken from the longest sequence's last one (the most keys) to the shortest's first, so that
    // what is left at the end is short: in order of the sequences alone eight ragged chunks took 4 % longer.
    // More than kSorted sequences are taken from the last to the first.
    volatile int* order = reinterpret_cast<int*>(sm + PS_ORDER);  // sequences by falling length
    volatile int* start = reinterpret_cast<int*>(sm + PS_START);  // blocks before each, and in all
    volatile int* len = reinterpret_cast<int*>(sm + PS_LEN);
    const bool sorted = a.N <= kSorted;
    if (tid == 0) {
        ctrl[1] = -1;
        ctrl[5] = 0;
    }
    if (sorted) {
        bool bad = false;
        int b = 0, mine = -1;
        if (tid < a.N) {
            b = blocks_of(tid, bad);
            mine = bad ? -1 : a.cu_k[tid + 1] - a.cu_k[tid];
            len[tid] = mine;
            if (bad && blockIdx.x == 0) report(a.dev_status, KDA_DEV_BAD_SEQLEN);
        }
        __syncthreads();
        if (tid < a.N) {
            int rank_of = 0;
            for (int m = 0; m < a.N; ++m) {
                const int x = len[m];
                rank_of += x > mine || (x == mine && m > tid);
            }
            order[rank_of] = tid;
            start[rank_of + 1] = b;
        }
        __syncthreads();
        if (warp == 0) {
            int before = 0;
            for (int base = 0; base < a.N; base += 32) {
                const int r = base + lane;
                int x = r < a.N ? start[r + 1] : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int z = __shfl_up_sync(~0u, x, o);
                    if (lane >= o) x += z;
                }
                if (r < a.N) start[r + 1] = before + x;
                before += __shfl_sync(~0u, x, 31);
            }
            if (lane == 0) start[0] = 0;
        }
        __syncthreads();
        if (tid < a.N && y >= start[tid] && y < start[tid + 1]) {
            ctrl[1] = order[tid];
            ctrl[2] = start[tid + 1] - 1 - y;
        }
    } else {
        int before = 0;
        for (int base = 0; base < a.N; base += kPreThreads) {
            __syncthreads();
            // from the last sequence to the first
            const int n = a.N - 1 - (base + tid);
            bool bad = false;
            const int b = n >= 0 ? blocks_of(n, bad) : 0;
            if (bad && blockIdx.x == 0) report(a.dev_status, KDA_DEV_BAD_SEQLEN);
            int x = b;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int z = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += z;
            }
            if (lane == 31) scan[warp] = x;
            __syncthreads();
            const int stood = before;
            int off = before;
            for (int w = 0; w < kPreThreads / 32; ++w) {
                if (w < warp) off += scan[w];
                before += scan[w];
            }
            const int lo = off + x - b;
            if (b > 0 && y >= lo && y < lo + b) {
                ctrl[1] = n;
                ctrl[2] = b - 1 - (y - lo);
                ctrl[3] = base;
                ctrl[4] = stood;
            }
            // block 0 looks at every sequence, for the report
            if (before > y && blockIdx.x != 0) break;
        }
    }
    __syncthreads();
    if (ctrl[1] < 0) return;
    if (tid < PB_BARS) {
        int count = 1;
        if (tid < PB_KFREE) count = 2;                          // an arrival of each CTA
        if (tid >= PB_P && tid < PB_O) count = 8;               // four warps of each
        if (tid >= PB_IFREE && tid < PB_DRAIN) count = rank == 0 ? 9 : 8;  // the warps that read a block's place
        mbar_init(bar(tid), count);
    }
    if (warp == 9) tmem2_alloc(sb + PS_CTRL, 512);
    // a block: its place, and the key tiles of its two query tiles (over both CTAs), up to the last key
    // that the tile's last row sees
    struct Block {
        int h, q0, Lq, k0, Lk, row0, n0, n1, nt;
    };
    auto block_at = [&](int h, int n, int row0) {
        Block u;
        u.h = h;
        u.row0 = row0;
        u.q0 = a.cu_q[n], u.Lq = a.cu_q[n + 1] - u.q0, u.k0 = a.cu_k[n], u.Lk = a.cu_k[n + 1] - u.k0;
        auto tiles_of = [&](int q) {
            const int rows = min(kQTile, u.Lq - row0 - q * kQTile);
            if (rows <= 0) return 0;
            const int keys = a.full ? u.Lk : min(u.Lk, u.Lk - u.Lq + row0 + q * kQTile + rows);
            return keys > 0 ? (keys + kKTile - 1) / kKTile : 0;
        };
        u.n0 = tiles_of(0), u.n1 = tiles_of(1), u.nt = max(u.n0, u.n1);
        return u;
    };
    fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are there
    fence_after();
    const uint32_t tmem = ctrl[0];
    bool dead = false;
    // A wait that runs out marks both CTAs of the pair and ends its role: rows of the block are NaN then (the
    // MMA warp may still finish a tile with operands that did not come), the other roles' waits run out too.
    auto give_up = [&] {
        dead = true;
        for (uint32_t c = 0; c < 2; ++c)
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(map_rank(sb + PS_CTRL + 20, c)), "r"(0x7fffffff) : "memory");
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        report(a.dev_status, KDA_DEV_TIMEOUT);
    };
    auto wait = [&](int b, uint32_t parity) {
        if (dead) return;
        if (!mbar_wait(bar(b), parity, kPreWait)) give_up();
    };

    if (warp == 8) {
        // ================================================================ loads
        // into this CTA, counted on the barriers of the first
        auto first = [&](int b) { return map_rank(bar(b), 0); };
        Block u = block_at((int)(blockIdx.x >> 1) % a.H, ctrl[1], ctrl[2] * kQBlock);
        uint32_t kt = 0, vt = 0, n_q[2] = {0, 0}, edges = 0;  // tiles, query tiles and edges loaded so far
        int scan_base = ctrl[3], scan_before = ctrl[4];
        auto load_queries = [&](int q) {
            if ((q ? u.n1 : u.n0) == 0) return;
            if (n_q[q] > 0) wait(PB_QFREE + q, (n_q[q] - 1) & 1);
            ++n_q[q];
            if (dead || lane != 0) return;
            mbar_expect_tx_cluster(first(PB_Q + q), 3 * kQPart);
            for (int c = 0; c < 3; ++c)
                tma2_load_3d(sb + (q * 3 + c) * kQPart, &maps.q, 64 * c, u.h * a.hq,
                             u.q0 + u.row0 + q * kQTile + (int)rank * kRows, first(PB_Q + q));
        };
        auto load_k = [&](int i) {
            const uint32_t st = kt % kStages;
            wait(PB_KFREE + st, (kt / kStages & 1) ^ 1);
            ++kt;
            if (dead || lane != 0) return;
            const int t = u.k0 + i * kKTile + (int)rank * 64;
            const uint32_t dst = sb + PS_K + st * kKBytes, b = first(PB_K + st);
            mbar_expect_tx_cluster(b, kKBytes);
            tma2_load_3d(dst, &maps.k, 0, u.h * a.hk, t, b);
            tma2_load_3d(dst + kKPart, &maps.k, 64, u.h * a.hk, t, b);
            tma2_load_2d(dst + 2 * kKPart, &maps.kr, 0, t, b);
        };
        auto load_v = [&](int i) {
            const uint32_t st = vt % kStages;
            wait(PB_VFREE + st, (vt / kStages & 1) ^ 1);
            if (kGiveUp && !dead && (int)blockIdx.x == a.give_up_cta && (int)vt == a.give_up_tile) give_up();
            ++vt;
            if (__any_sync(~0u, dead)) return;
            const uint32_t dst = sb + PS_V + st * kVBytes, b = first(PB_V + st);
            const int valid = u.Lk - i * kKTile;
            if (valid >= kKTile) {
                if (lane == 0) {
                    mbar_expect_tx_cluster(b, kVBytes);
                    tma2_load_3d(dst, &maps.v, 64 * (int)rank, u.h * a.hv, u.k0 + i * kKTile, b);
                }
            } else {
                // keys past the sequence (its last tile): their weight is zero, and so has to be the
                // value (what lies there belongs to another sequence).  This warp waits for the tile,
                // clears them and only then lets it be used.
                if (lane == 0) {
                    mbar_expect_tx(bar(PB_EDGE), kVBytes);
                    tma_load_3d(dst, &maps.v, 64 * (int)rank, u.h * a.hv, u.k0 + i * kKTile, bar(PB_EDGE));
                }
                wait(PB_EDGE, edges++ & 1);
                if (__any_sync(~0u, dead)) return;
                for (uint32_t e = valid * 128 + lane * 16; e < kVBytes; e += 512)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(dst + e), "r"(0u) : "memory");
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(b);
            }
        };
        // The place of block `id` of the grid: heads side by side.  Answers come in rising order, so the scan
        // over many sequences goes on where it stood (and starts again if one should not).
        auto place = [&](int id, int& n, int& row0) {
            const int want = id / a.H;
            n = -1;
            if (sorted) {
                for (int base = 0; base < a.N; base += 32) {
                    const int r = base + lane;
                    const uint32_t hit = __ballot_sync(~0u, r < a.N && want >= start[r] && want < start[r + 1]);
                    if (hit) {
                        const int at = base + __ffs(hit) - 1;
                        n = order[at];
                        row0 = (start[at + 1] - 1 - want) * kQBlock;
                        return;
                    }
                }
                return;
            }
            if (want < scan_before) scan_base = scan_before = 0;
            for (; scan_base < a.N; scan_base += 32) {
                const int c = a.N - 1 - (scan_base + lane);
                bool bad = false;
                const int b = c >= 0 ? blocks_of(c, bad) : 0;
                int x = b;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int z = __shfl_up_sync(~0u, x, o);
                    if (lane >= o) x += z;
                }
                const int lo = scan_before + x - b, total = __shfl_sync(~0u, x, 31);
                const uint32_t hit = __ballot_sync(~0u, b > 0 && want >= lo && want < lo + b);
                if (hit) {
                    const int who = __ffs(hit) - 1;
                    n = __shfl_sync(~0u, c, who);
                    row0 = __shfl_sync(~0u, b - 1 - (want - lo), who) * kQBlock;
                    return;
                }
                scan_before += total;
            }
        };
        for (uint32_t it = 0;; ++it) {
            // The next block is asked for under this one's last tiles, once both CTAs have read the last answer:
            // the pair that comes to its end first gets the next block.  (Asked for at a block's start, the
            // first pairs to start got them all: 8192 tokens at 8 heads 142 us for 106, 4096 at 16 heads 82 for 64.)
            auto ask = [&] {
                if (rank == 0 && it > 0) wait(PB_NEXT, (it - 1) & 1);
                if (lane == 0 && !dead) {
                    mbar_expect_tx(bar(PB_CLC), 16);
                    if (rank == 0) clc_request(sb + PS_CLC, bar(PB_CLC));
                }
                __syncwarp();
            };
            load_queries(0);
            if (u.nt > 0) load_k(0);
            load_queries(1);
            if (u.nt < kAskTiles) ask();
            for (int i = 0; i < u.nt; ++i) {
                if (i == u.nt - kAskTiles) ask();
                load_v(i);
                if (i + 1 < u.nt) load_k(i + 1);
                if (__any_sync(~0u, dead)) break;
            }
            wait(PB_CLC, it & 1);
            if (__any_sync(~0u, dead)) break;
            const int got = clc_block(sb + PS_CLC);
            fence_async_smem();  // the answer has been read before the next one is written
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(first(PB_NEXT));
            int n = -1, row0 = 0;
            if (got >= 0) place(got >> 1, n, row0);
            // the place for the other warps (their first block is the CTA's own)
            const uint32_t b = it & 1;
            if (it >= 2) wait(PB_IFREE + b, ((it - 2) >> 1) & 1);
            const int h = got >= 0 ? (got >> 1) % a.H : 0;
            if (lane == 0) {
                info[8 * b] = h;
                info[8 * b + 1] = n;
                info[8 * b + 2] = row0;
                mbar_arrive(bar(PB_INFO + b));
            }
            __syncwarp();
            if (n < 0) break;
            u = block_at(h, n, row0);
        }
    } else if (warp == 9 && rank == 0) {
        // ================================================================ MMAs
        // the whole warp runs this, one lane issues (umma.cuh, mma_by)
        const uint32_t lead = elect_lane();
        const uint32_t sb4 = (sb & 0x3ffffu) >> 4;
        const uint32_t tm = __shfl_sync(~0u, tmem, 0);
        const uint32_t ids = idesc_16(DT == KDA_F16, 256, kKTile, false, false, a.negate);
        const uint32_t idv = idesc_16(DT == KDA_F16, 256, 128, false, true, false);
        uint32_t kv = 0, n_q[2] = {0, 0}, n_p[2] = {0, 0};  // K / V tiles, query tiles, products of S so far
        auto do_s = [&](int q, uint32_t st) {
            const uint32_t b4 = sb4 + PS_K / 16 + st * (kKBytes / 16);
#pragma unroll
            for (int c = 0; c < 3; ++c)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma2_by(lead, tm + PT_S + q * 128, desc_k4(sb4 + (q * 3 + c) * (kQPart / 16), 128, s),
                            desc_k4(b4 + c * (kKPart / 16), 64, s), ids, c + s != 0);
            commit2_by(lead, bar(PB_S + q));
        };
        auto do_pv = [&](int q, uint32_t st, int fresh, int s0, int s1) {
            const uint32_t b4 = sb4 + PS_V / 16 + st * (kVBytes / 16);
#pragma unroll
            for (int s = s0; s < s1; ++s)
                mma2_ta_by(lead, tm + PT_O + q * 128, tm + PT_S + q * 128 + 8 * s, desc_mn4(b4, 16, 1024, s), idv,
                           !fresh || s != 0);
            if (s1 == 8) commit2_by(lead, bar(PB_O + q));
        };
        Block u = block_at((int)(blockIdx.x >> 1) % a.H, ctrl[1], ctrl[2] * kQBlock);
        bool stop = false;
        for (uint32_t it = 0; !stop; ++it) {
            const int m0 = __shfl_sync(~0u, u.n0, 0), m1 = __shfl_sync(~0u, u.n1, 0), mt = max(m0, m1);
            if (mt > 0) wait(PB_K + kv % kStages, kv / kStages & 1);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int mq = q ? m1 : m0;
                if (mq > 0) {
                    wait(PB_Q + q, n_q[q]++ & 1);
                    fence_after();
                    do_s(q, kv % kStages);
                    if (mq == 1) commit2_by(lead, bar(PB_QFREE + q));
                }
            }
            if (mt > 0) commit2_by(lead, bar(PB_KFREE + kv % kStages));
            for (int i = 0; i < mt && !stop; ++i, ++kv) {
                const uint32_t st = kv % kStages, sn = (kv + 1) % kStages;
                // loads ahead of the weights: a wait queues behind the MMAs issued before it
                if (!mbar_wait_cluster(bar(PB_V + st), kv / kStages & 1, kPreWait)) give_up();  // cleared edges
                if (i + 1 < mt) wait(PB_K + sn, (kv + 1) / kStages & 1);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int mq = q ? m1 : m0, mo = q ? m0 : m1;
                    if (i < mq) {
                        wait(PB_P + q, n_p[q] & 1);
                        fence_after();
                        do_pv(q, st, i == 0, 0, 6);
                        wait(PB_P2 + q, n_p[q]++ & 1);
                        fence_after();
                        do_pv(q, st, 0, 6, 8);
                        if (q == 1 || i >= mo) commit2_by(lead, bar(PB_VFREE + st));
                        if (i + 1 < mq) {
                            do_s(q, sn);
                            if (i + 2 == mq) commit2_by(lead, bar(PB_QFREE + q));  // the last S that reads these queries
                            if (q == 1 || i + 1 >= mo) commit2_by(lead, bar(PB_KFREE + sn));
                        }
                    }
                }
                stop = __any_sync(~0u, dead);
            }
            if (stop) break;
            const uint32_t b = it & 1;
            wait(PB_INFO + b, (it >> 1) & 1);
            stop = __any_sync(~0u, dead);
            const int h = info[8 * b], n = info[8 * b + 1], row0 = info[8 * b + 2];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(PB_IFREE + b));
            stop = stop || __any_sync(~0u, n < 0);
            if (!stop) u = block_at(h, n, row0);
        }
        commit2_by(lead, bar(PB_DRAIN));
        dead = false;
        wait(PB_DRAIN, 0);
    } else if (warp < 8) {
        // ================================================================ softmax and results
        const int q = warp >> 2, t = tid & 127;
        const uint32_t tq = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = tq + PT_S + q * 128, to = tq + PT_O + q * 128;
        const uint32_t p_full = map_rank(bar(PB_P + q), 0), p_full2 = map_rank(bar(PB_P2 + q), 0);
        uint32_t done = 0;  // key tiles of this query tile so far
        Block u = block_at((int)(blockIdx.x >> 1) % a.H, ctrl[1], ctrl[2] * kQBlock);
        for (uint32_t it = 0;; ++it) {
            const int my_tiles = q ? u.n1 : u.n0;
            const int row = u.row0 + q * kQTile + (int)rank * kRows + t;  // of the sequence
            const int last = row >= u.Lq ? -1 : a.full ? u.Lk - 1 : u.Lk - u.Lq + row;
            float m = -inf;
            // in shared memory: two registers more across a tile spill others (837 us for 775, eight chunks)
            WeightSum* sum = reinterpret_cast<WeightSum*>(sm + PS_SUM) + tid;
            *sum = WeightSum();
            for (int i = 0; i < my_tiles && !__any_sync(~0u, dead); ++i, ++done) {
                uint32_t s[4][32];
                wait(PB_S + q, done & 1);
                fence_after();
#pragma unroll
                for (int b = 0; b < 4; ++b) ld32_issue(ts + 32 * b, s[b]);
                wait_ld();
                const int lim = last - i * kKTile;  // columns 0 .. lim are seen
                if (lim < kKTile - 1) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * b + e > lim) s[b][e] = __float_as_uint(-inf);
                }
                float mx[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) mx[k] = __uint_as_float(s[k >> 1][k & 1]);
#pragma unroll
                for (int e = 2; e < 32; e += 4)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(s[k >> 1][e + (k & 1)])),
                                      __uint_as_float(s[k >> 1][(e + 2 + (k & 1)) & 31]));
                const float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                       fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
                float f = 1.f;
                bool need = false;
                if (i == 0) {
                    m = mt;
                } else if (mt > m && (m == -inf || (mt - m) * a.c > 8.f)) {
                    f = ex2((m - mt) * a.c);
                    m = mt;
                    need = true;
                }
                if (__any_sync(~0u, need)) {
                    wait(PB_O + q, (done - 1) & 1);
                    fence_after();
#pragma unroll 1
                    for (int b = 0; b < 8; ++b) {
                        float o[16];
                        ld16(to + 16 * b, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= f;
                        st16f(to + 16 * b, o);
                    }
                    sum->scale(f);
                }
                const float mc = m == -inf ? 0.f : log2_base<DT>(m, a.c);
                const float2 cc = make_float2(a.c, a.c), nm = make_float2(-mc, -mc);
                float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 x = __ffma2_rn(make_float2(__uint_as_float(s[b][2 * e]), __uint_as_float(s[b][2 * e + 1])), cc, nm);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        ls[e & 1] = __fadd2_rn(ls[e & 1], x);
                        p[e] = E::put2(x.x, x.y);
                    }
                    st16u(ts + 16 * b, p);
                    // the first 96 keys go ahead: their product runs under the last exponentials
                    if (b >= 2) {
                        wait_st();
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(b == 2 ? p_full : p_full2);
                    }
                }
                sum->add((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y));
            }
            if (my_tiles > 0) {
                wait(PB_O + q, (done - 1) & 1);
                fence_after();
            }
            float gone;  // 0, or NaN after a wait ran out; by its address: as ctrl[5] the tile loop spilled (1 % slower)
            asm volatile("ld.volatile.shared.f32 %0, [%1];" : "=f"(gone) : "r"(sb + PS_CTRL + 20) : "memory");
            const float l = sum->total() + gone, il = 1.f / l;
            const int64_t orow = (int64_t)u.q0 + row;
            if (row < u.Lq && a.lse != nullptr)
                a.lse[orow * a.H + u.h] = l == 0.f ? -inf : (log2_base<DT>(m, a.c) + log2f(l)) * 0.69314718055994531f;
            const int64_t at = orow * a.out_rs + (int64_t)u.h * a.out_hs;
            // a thread's row, whole 32-byte sectors at a time; the other query tile's products go on meanwhile
            auto emit = [&](auto put) {
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    float o[32];
                    if (my_tiles > 0) {
                        ld32(to + 32 * b, o);
                        // a row without keys is zero by choice, not by its factor: beside a NaN or infinity
                        // that other rows see, its sums are NaN
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0.f : o[e] * il;
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.f;
                    }
                    if (row < u.Lq) put(o, 32 * b);
                }
            };
            if (a.out_dt == KDA_F32) {
                float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
                emit([&](const float (&o)[32], int c) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) p[(c + e) / 4] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                });
            } else if (a.out_dt == KDA_BF16) {
                uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at);
                emit([&](const float (&o)[32], int c) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) p[(c + e) / 8] = pack16<KDA_BF16>(o, e);
                });
            } else {
                uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at);
                emit([&](const float (&o)[32], int c) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) p[(c + e) / 8] = pack16<KDA_F16>(o, e);
                });
            }
            fence_before();
            const uint32_t b = it & 1;
            wait(PB_INFO + b, (it >> 1) & 1);
            if (__any_sync(~0u, dead)) break;
            const int h = info[8 * b], n = info[8 * b + 1], row0 = info[8 * b + 2];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(PB_IFREE + b));
            if (n < 0) break;
            u = block_at(h, n, row0);
        }
    }
    fence_before();
    __syncthreads();
    // Every load and answer was waited for by a role that is done.  After a wait that ran out that does not
    // hold: a bounded wait on a barrier that nothing arrives on (about a second) lets them land.
    if (ctrl[5] && warp == 8) {
        mbar_wait(bar(PB_NEVER), 0, kPreWait);
        __syncwarp();
    }
    cluster_sync();  // no CTA leaves while the other's MMAs, loads or arrivals may still reach it
    fence_after();
    if (warp == 9) tmem2_dealloc(tmem, 512);
}

// Tensor map over rows of heads: (channel, head, row), one box 64 channels of one head.
bool rows_map(CUtensorMap* map, kda_dtype dt, const LatentRows& r, int channels, int H, int T, int rows) {
    // a dimension that is not stepped along (one head or row, or heads that share a row) has size 1
    // and any legal stride
    const cuuint64_t dims[3] = {(cuuint64_t)channels, (cuuint64_t)(r.hs ? H : 1), (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)(r.hs ? r.hs : channels) * 2, (cuuint64_t)(r.rs ? r.rs : channels) * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    return encode_16bit(map, dt, 3, r.base, dims, strides, box);
}

}  // namespace
}  // namespace kda

using namespace kda;

namespace kda {
namespace {

// Both entry points; give_up_cta < 0 for the call itself.
kda_status prefill_call(const kda_rows_desc* q, const kda_rows_desc* k_nope, const void* k_rope, int64_t k_rope_stride,
                        const kda_rows_desc* v, kda_dtype in_dtype, const int32_t* cu_q, const int32_t* cu_k, int32_t N,
                        int32_t Tq, int32_t Tk, int32_t H, int32_t d_nope, int32_t d_rope, int32_t dv, float scale,
                        uint32_t flags, const kda_rows_desc* out, kda_dtype out_dtype, float* lse, int32_t* dev_status,
                        void* stream, int32_t give_up_cta, int32_t give_up_tile) {
    KDA_REQUIRE(N >= 0 && Tq >= 0 && Tk >= 0 && H > 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(d_nope == kNope && d_rope == kRope && dv == kHeadV, KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((in_dtype == KDA_BF16 || in_dtype == KDA_F16) && any_dtype_ok(out_dtype), KDA_ERR_UNSUPPORTED);
    KDA_REQUIRE((flags & ~KDA_LATENT_FULL) == 0, KDA_ERR_UNSUPPORTED);
    const int64_t blocks = ((int64_t)Tq / kQBlock + N) * H;
    KDA_REQUIRE(blocks < (1ll << 30) && Tk < (1 << 30) && Tq < (1 << 30), KDA_ERR_UNSUPPORTED);
    if (N == 0 || Tq == 0) return KDA_OK;
    KDA_REQUIRE(isfinite(scale), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(rows_ok(q) && rows_ok(out), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(k_nope != nullptr && v != nullptr, KDA_ERR_INVALID_ARG);
    if (Tk > 0) {
        KDA_REQUIRE(rows_ok(k_nope) && rows_ok(v), KDA_ERR_INVALID_ARG);
        KDA_REQUIRE(k_rope != nullptr && aligned16(k_rope), KDA_ERR_INVALID_ARG);
    }
    const kda_rows_desc* ds[] = {q, k_nope, v, out};
    for (const kda_rows_desc* d : ds) KDA_REQUIRE(d->row_stride >= 0 && d->head_stride >= 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE((q->row_stride > 0 || Tq == 1) && ((k_nope->row_stride > 0 && v->row_stride > 0) || Tk <= 1),
                KDA_ERR_INVALID_ARG);
    const void* ptrs[] = {cu_q, cu_k};
    for (const void* p : ptrs) KDA_REQUIRE(p != nullptr && aligned16(p), KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(k_rope_stride % 8 == 0 && k_rope_stride >= kRope, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(aligned16(lse) && aligned16(dev_status), KDA_ERR_INVALID_ARG);
    PreMaps maps;
    const LatentRows rq = as_rows(q), rk = Tk > 0 ? as_rows(k_nope) : rq, rv = Tk > 0 ? as_rows(v) : rq;
    KDA_REQUIRE(rows_map(&maps.q, in_dtype, rq, kHeadK, H, Tq, 128), KDA_ERR_CUDA);
    if (Tk > 0) {
        KDA_REQUIRE(rows_map(&maps.k, in_dtype, rk, kNope, H, Tk, 64), KDA_ERR_CUDA);
        KDA_REQUIRE(rows_map(&maps.v, in_dtype, rv, kHeadV, H, Tk, 128), KDA_ERR_CUDA);
        const cuuint64_t dims[2] = {kRope, (cuuint64_t)Tk};
        const cuuint64_t strides[1] = {(cuuint64_t)k_rope_stride * 2};
        const cuuint32_t box[2] = {64, 64};
        KDA_REQUIRE(encode_16bit(&maps.kr, in_dtype, 2, k_rope, dims, strides, box), KDA_ERR_CUDA);
    } else {
        maps.k = maps.kr = maps.v = maps.q;  // no key, no load
    }
    const PrefillArgs a{cu_q, cu_k, N, Tq, Tk, H, rq.hs != 0, rk.hs != 0, rv.hs != 0, log2_scale(scale), scale < 0.f,
                        (flags & KDA_LATENT_FULL) != 0, const_cast<void*>(out->base), out->row_stride, out->head_stride,
                        out_dtype, lse, dev_status, give_up_cta, give_up_tile};
    auto* f = give_up_cta >= 0       ? prefill_kernel<KDA_BF16, true>
              : in_dtype == KDA_BF16 ? prefill_kernel<KDA_BF16, false>
                                     : prefill_kernel<KDA_F16, false>;
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PS_SMEM) != cudaSuccess)
        return runtime_failed();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks * 2);
    cfg.blockDim = dim3(kPreThreads);
    cfg.dynamicSmemBytes = PS_SMEM;
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, f, maps, a) != cudaSuccess) return runtime_failed();
    return launch_status();
}

}  // namespace
}  // namespace kda

extern "C" kda_status kda_latent_prefill(const kda_rows_desc* q, const kda_rows_desc* k_nope,
                                         const void* k_rope, int64_t k_rope_stride,
                                         const kda_rows_desc* v, kda_dtype in_dtype,
                                         const int32_t* cu_q, const int32_t* cu_k, int32_t N,
                                         int32_t Tq, int32_t Tk, int32_t H, int32_t d_nope,
                                         int32_t d_rope, int32_t dv, float scale, uint32_t flags,
                                         const kda_rows_desc* out, kda_dtype out_dtype, float* lse,
                                         int32_t* dev_status, void* stream) {
    return prefill_call(q, k_nope, k_rope, k_rope_stride, v, in_dtype, cu_q, cu_k, N, Tq, Tk, H, d_nope, d_rope, dv, scale, flags,
                        out, out_dtype, lse, dev_status, stream, -1, 0);
}

extern "C" kda_status kda_selftest_latent_prefill_give_up(
    const kda_rows_desc* q, const kda_rows_desc* k_nope, const void* k_rope, int64_t k_rope_stride, const kda_rows_desc* v,
    kda_dtype in_dtype, const int32_t* cu_q, const int32_t* cu_k, int32_t N, int32_t Tq, int32_t Tk, int32_t H,
    int32_t d_nope, int32_t d_rope, int32_t dv, float scale, uint32_t flags, const kda_rows_desc* out, kda_dtype out_dtype,
    float* lse, int32_t* dev_status, void* stream, int32_t block, int32_t tile) {
    KDA_REQUIRE(block >= 0 && tile >= 0, KDA_ERR_INVALID_ARG);
    KDA_REQUIRE(in_dtype == KDA_BF16, KDA_ERR_UNSUPPORTED);
    return prefill_call(q, k_nope, k_rope, k_rope_stride, v, in_dtype, cu_q, cu_k, N, Tq, Tk, H, d_nope, d_rope, dv, scale, flags,
                        out, out_dtype, lse, dev_status, stream, block, tile);
}
