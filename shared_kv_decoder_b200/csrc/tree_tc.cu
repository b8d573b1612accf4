// Attention of drafted tokens on the sm_100a tensor cores (bf16 in, fp32
// softmax and accumulation): the work of tree.cuh with 128-key tiles.
//
// The rows of one KV head -- every node's query heads of that group, row =
// node * G + head -- are the M rows of S = Q K^T and O += P V, so one read of
// the context serves all drafted tokens.  Two layouts:
//   ALT   N * G <= 128: one 128-row tile, and the stream's KV tiles alternate
//         between two softmax warpgroups, each with its own S / P and O and its
//         own running maximum; they are added up when the segment ends.
//   PAIR  more rows: two row tiles (256 rows) read the same KV tile.
// Either way the tensor core works for one softmax chain while the other's
// exponentials run.
//
// What bounds it.  With R rows of a KV head a 64 KB K / V tile (D = 128) takes
// 4 * 128 * max(R, 128) * 128 tensor operations; at the measured rates the cache
// read is the longer one up to about R = 250.  Measured (graph replays on
// several GPUs): 16 x 64K-128K tokens, 16 nodes (R = 64): 930-1075 us,
// 5.9-6.8 TB/s of the cache, the clock at 1.3-1.5 GHz under the power cap;
// 131007 tokens, 64 nodes (R = 256): 159-179 us, 768-865 TFLOP/s, the chain of
// one tile's softmax (1850 cycles) and the MMAs that wait for it (about 2000) the
// limit, tensor pipe half busy; 64 x 48 nodes over the 1024 ring: 117-120 us, a
// segment's start and end (nine tiles) a quarter of it; in clusters 2047 tokens
// 10.5 us, 4 x 16 nodes over the ring 12.8, latency throughout.  One warp has a
// whole row, so that nothing is agreed on between warps, and all exponentials
// are MUFU's.
//
// Warp roles (384 threads):
//   warps 0-3, 4-7  softmax chains A and B: thread r owns row r (TMEM lane r)
//   warps 8, 10     TMA, one thread each (a warp of its own, so that one's wait never
//                   holds up the other's copies).  PAIR: K, and Q and V.  ALT: Q and
//                   chain A's K and V, and chain B's: each chain has a ring of its
//                   own whose stages take K, V, K, V, ... in turn, and waits for
//                   every one of them, so no parity can mean an older phase
//   warps 9, 11     MMA issue of chain A and of chain B, one thread each: a wait or
//                   a commit takes about a hundred cycles of its thread even when
//                   nothing is left to wait for, and with one thread for both
//                   chains these, not the tensor core, set the pace
// TMEM (512 columns): S_A/P_A, S_B/P_B, O_A, O_B, 128 columns each; P is bf16
// over the first 64 columns of its S.
//
// Masks.  Only a tile that some row does not see whole is masked, by one bit a
// column.  The product with V needs more: a weight of 0 times an infinity is
// NaN, so in such a tile the V rows that no row sees are cleared in shared
// memory before P V, and so are the infinities and NaN of rows that some row
// may see -- those are then added to the outputs of the rows that do see them
// when the segment ends (a path that finite inputs never take).
//
// Every mbarrier wait is bounded; a wait that gives up sets the status word,
// and all roles fall through to the common exit, which waits for issued copies
// and MMAs before freeing TMEM.
#include <cuda.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "cluster.cuh"
#include "common.cuh"
#include "launch.h"
#include "tc.cuh"
#include "tree.cuh"

namespace yoco {

// Bit 0: a bounded wait gave up; bit 1: a sequence's arguments were out of range.
static __device__ unsigned int g_status_tree_tc;

namespace tree {
namespace {

constexpr int BN = kTcKeys;
constexpr int kThreads = 384;
// Registers of a thread: at the launch, of a warp that copies or issues, of a softmax warp.
constexpr int kRegs = 168, kFewRegs = 72, kManyRegs = 216;
static_assert(128 * kFewRegs + 256 * kManyRegs <= kThreads * kRegs, "no more than the launch has");
constexpr int kTmemCols = 512;
constexpr uint32_t kBlk = 128 * 128;   // one [128 rows x 128 bytes] swizzled block

template <int D, bool PAIR>
struct Smem {
    static constexpr int KB = D / 64;
    static constexpr uint32_t TILE = (uint32_t)KB * kBlk;
    static constexpr int QTILES = PAIR ? 2 : 1;
    // stages: of K and of V (PAIR), of chain A's ring and of chain B's (ALT)
    static constexpr int KST = D == 128 ? 3 : 6;
    static constexpr int VST = (D == 128 ? 3 : 6) - (PAIR ? 1 : 0);
    static constexpr uint32_t Q = 0;
    static constexpr uint32_t K = Q + QTILES * TILE;
    static constexpr uint32_t V = K + KST * TILE;
    static constexpr uint32_t ML = V + VST * TILE;      // float2[128]: chain B's (m, l)
    static constexpr uint32_t BAR = ML + 128 * 8;
    static constexpr uint32_t MISC = BAR + 50 * 8;
    static constexpr uint32_t BYTES = MISC + 256;
    static constexpr uint32_t ALLOC = BYTES + 1024;     // alignment slack
};
static_assert(Smem<128, true>::ALLOC <= 232448 && Smem<128, false>::ALLOC <= 232448, "shared memory");

enum Bar {
    kQFull = 0,    // 2: Q tile loaded
    kQEmpty = 2,   // 2: last S MMA on the Q tile done
    kSFull = 4,    // 2: S of chain A / B ready
    kPFull = 6,    // 2: P written (4 arrivals, one a warp)
    kODone = 8,    // 2: P.V finished
    kOFree = 10,   // 2: O read out (4 arrivals)
    kML = 12,      // ALT: chain B's (m, l) written; PAIR in clusters: its last P V seen to finish (4 arrivals)
    kDrain = 13,   // 2
    kKFull = 15,   // up to 6 each; ALT: of chain A's ring
    kKEmpty = 21,
    kVFull = 27,   // ALT: of chain B's ring
    kVEmpty = 33,
    kVClean = 39,  // PAIR: chain A is done with cleaning the tile (4 arrivals)
    kTurn = 45,    // 2: chain A's / B's turn to issue MMAs
    kPHalf = 47,   // 2: the first 64 columns of P written (4 arrivals)
    kNumBars = 49
};

struct Misc {
    uint32_t tmem;
    int abort;
    ClusterIter share;
    Seq seq;
    int poison[8];   // by segment mod 8: the last segment with an infinity or NaN cleared from a seen V row
    Range range;
};
static_assert(sizeof(Misc) <= 256, "misc area");

YOCO_DEV bool wait1(uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, &g_status_tree_tc); }
YOCO_DEV bool waitw(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, &g_status_tree_tc));
}

// The two bf16 of w that are infinite or NaN (an exponent of all ones), as
// their sign bits: adding the lowest exponent bit carries into them.
YOCO_DEV uint32_t odd_bits(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
YOCO_DEV uint32_t clear_odd(uint32_t w) {
    const uint32_t t = odd_bits(w);
    return w & ~((t >> 15 & 1u) * 0xffffu | (t >> 31) * 0xffff0000u);
}

// Chunks [c0, c0 + NC) of each 64-column block of key row r of a V tile: cleared
// (unseen), or cleared of its infinities and NaN; true when there were any of
// those.  Chunks by the swizzle's order, which keeps a quarter-warp off one bank
// group.
template <int KB, int NC>
YOCO_DEV bool clean_v_row(uint8_t *tile, int r, int c0, bool unseen) {
    uint8_t *row = tile + r * 128;
    auto at = [&](int i) {
        return reinterpret_cast<uint4 *>(row + i / NC * kBlk + (((c0 + i % NC) ^ (r & 7)) << 4));
    };
    if (unseen) {
#pragma unroll 4
        for (int i = 0; i < NC * KB; ++i) *at(i) = make_uint4(0, 0, 0, 0);
        return false;
    }
    uint32_t odd = 0;
#pragma unroll 4
    for (int i = 0; i < NC * KB; ++i) {
        const uint4 v = *at(i);
        odd |= odd_bits(v.x) | odd_bits(v.y) | odd_bits(v.z) | odd_bits(v.w);
    }
    if (odd) {
        for (int i = 0; i < NC * KB; ++i) {
            const uint4 v = *at(i);
            *at(i) = make_uint4(clear_odd(v.x), clear_odd(v.y), clear_odd(v.z), clear_odd(v.w));
        }
    }
    return odd != 0;
}

// 32-byte global store, not kept in L1; the address a multiple of 32.
YOCO_DEV void st_global_32B(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// The infinities and NaN of one seen V row, added to 32 columns of its output.
YOCO_DEV void add_odd(const __nv_bfloat16 *v, float *o) {
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
        float f[8];
        Chunk<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(v + e), f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!isfinite(f[i])) o[e + i] += f[i];
    }
}

// The larger of three, NaN if any is.
YOCO_DEV float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A ring segment's bounds over all its nodes: what every node sees and what
// any does.
struct RingSpan {
    RingBounds every, any;
};

}  // namespace

template <int D, bool RING, bool PAIR, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kn,
                   const __grid_constant__ CUtensorMap tm_vn, const __grid_constant__ Params p) {
    using L = Smem<D, PAIR>;
    constexpr int KB = L::KB;
    constexpr int RS = PAIR ? 256 : 128;
    using Iter = std::conditional_t<CLUSTER, ClusterIter, SegIter<RING, RS, BN>>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *sbase = smem_raw + (base - raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sbase + L::BAR);
    Misc *misc = reinterpret_cast<Misc *>(sbase + L::MISC);
    volatile int *abort_flag = &misc->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_trigger();
    if (threadIdx.x == 32) {
        tc::prefetch_map(&tm_q);
        tc::prefetch_map(&tm_k);
        tc::prefetch_map(&tm_v);
        tc::prefetch_map(&tm_kn);
        tc::prefetch_map(&tm_vn);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars[kQFull + s], 1);
            mbar_init(&bars[kQEmpty + s], PAIR ? 1 : 2);   // ALT: both chains read the one tile
            mbar_init(&bars[kSFull + s], 1);
            mbar_init(&bars[kPFull + s], 4);
            mbar_init(&bars[kPHalf + s], 4);
            mbar_init(&bars[kODone + s], 1);
            mbar_init(&bars[kOFree + s], 4);
            mbar_init(&bars[kTurn + s], 1);
        }
        mbar_init(&bars[kML], 4);
        for (int s = 0; s < 2; ++s) mbar_init(&bars[kDrain + s], 1);
        for (int s = 0; s < 6; ++s) {
            mbar_init(&bars[kKFull + s], 1);
            mbar_init(&bars[kKEmpty + s], PAIR ? 2 : 1);   // PAIR: both chains read the tile
            mbar_init(&bars[kVFull + s], 1);
            mbar_init(&bars[kVEmpty + s], PAIR ? 2 : 1);
            mbar_init(&bars[kVClean + s], 4);
        }
        misc->abort = 0;
        for (int s = 0; s < 8; ++s) misc->poison[s] = -1;
        fence_mbar_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(&misc->tmem, kTmemCols);
        tc::tmem_relinquish();
    }
    pdl_wait();
    if (warp == 8) {
        // once any CTA has recorded a timeout, the rest of the grid does nothing
        const bool idle = *(volatile unsigned int *)&g_status_tree_tc & 1u;
        if constexpr (CLUSTER) {
            if (lane == 0) {
                Seq q;
                ClusterIter s = cluster_share<RING, RS, BN>(p, (int)blockIdx.x / p.cluster, (int)blockIdx.x % p.cluster,
                                                            p.cluster, &q);
                if (idle) s.any = false;
                misc->share = s;
                misc->seq = q;
                if (!q.ok && s.s.g == 0 && s.s.rt == 0) atomicOr(&g_status_tree_tc, kStatusBadSequence);
            }
        } else {
            find_range<RING, RS, BN>(p, &misc->range);
            if (lane == 0 && idle) misc->range.x = misc->range.end;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = misc->tmem;
    auto segments = [&] {
        if constexpr (CLUSTER) return misc->share;
        else return Iter(p, misc->range);
    };

    // registers: 384 x 168 at the launch, 128 x 72 + 256 x 216 from here (with 168 for
    // all, 159 us for the 120 of 64 x 48 nodes over the 1024 ring, 180 for the 160 of
    // 64 nodes over 131007 tokens)
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == 8 || warp == 10) {
            // ----------------------------------------------------- TMA producers
            Iter it = segments();
            Seg sg;
            const bool one = warp == 8;                     // K / chain A
            const int ST = one ? L::KST : L::VST;
            uint64_t *full = &bars[one ? kKFull : kVFull], *empty = &bars[one ? kKEmpty : kVEmpty];
            int u = 0, k = 0;   // copies, segments whose Q is on its way
            if (lane == 0) {
                const bool has_q = PAIR ? !one : one;
                const uint32_t dst0 = base + (one ? L::K : L::V);
                bool ok = true;
                while (ok && !*abort_flag && it.next(p, sg)) {
                    if (has_q) {
                        for (int hh = 0; hh < L::QTILES && ok; ++hh) {
                            ok = wait1(&bars[kQEmpty + hh], (k & 1) ^ 1);
                            if (!ok) break;
                            mbar_arrive_expect_tx(&bars[kQFull + hh], 128 * D * 2);
                            const int node0 = (sg.rt * L::QTILES + hh) * (128 >> p.lg);
                            for (int kb = 0; kb < KB; ++kb)
                                tc::tma_load_4d(base + L::Q + hh * L::TILE + kb * kBlk, &tm_q, kb * 64, sg.g << p.lg, node0,
                                                sg.b, &bars[kQFull + hh]);
                        }
                        if (ok) ++k;
                    }
                    for (int t = sg.t0 + (PAIR || one ? 0 : 1); ok && t < sg.t1; t += PAIR ? 1 : 2) {
                        const bool nodes = t == sg.n_ctx_tiles;
                        const int row = nodes ? 0 : RING ? t * BN : (int)(sg.row0 + (int64_t)t * BN);
                        const int b = nodes || RING ? sg.b : 0;
#pragma unroll
                        for (int e = 0; e < (PAIR ? 1 : 2) && ok; ++e) {
                            const bool is_k = PAIR ? one : e == 0;
                            const CUtensorMap *map = is_k ? nodes ? &tm_kn : &tm_k : nodes ? &tm_vn : &tm_v;
                            const int st = u % ST;
                            ok = wait1(&empty[st], ((u / ST) & 1) ^ 1);
                            if (!ok) break;
                            mbar_arrive_expect_tx(&full[st], (nodes ? kTreeMaxNodes : BN) * D * 2);
                            for (int kb = 0; kb < KB; ++kb)
                                tc::tma_load_4d(dst0 + st * L::TILE + kb * kBlk, map, kb * 64, sg.g, row, b, &full[st]);
                            ++u;
                        }
                    }
                }
                if (!ok) *abort_flag = 1;
            }
            __syncwarp();
            // with every copy issued, these warps have time
            if (!CLUSTER) fill_rows_without_node<__nv_bfloat16, D, RING, RS, BN>(p, warp == 10, 2, &g_status_tree_tc);
            if (lane == 0) {
                // drain: the last copies issued must land before this CTA may exit
                for (int q = max(0, u - ST); q < u; ++q)
                    if (!wait1(&full[q % ST], (q / ST) & 1)) break;
                if (k > 0)
                    for (int hh = 0; hh < L::QTILES; ++hh)
                        if (!wait1(&bars[kQFull + hh], (k - 1) & 1)) break;
            }
        } else {
            // ------------------------------------------- MMA issue of one chain
            if (lane == 0) {
                Iter it = segments();
                Seg sg;
                const int hh = warp == 9 ? 0 : 1;
                constexpr uint32_t idS = tc::idesc_bf16(128, BN, false, false);
                constexpr uint32_t idPV = tc::idesc_bf16(128, D, false, true);
                // descriptors as (low, high) words: the low one holds the address and the
                // leading offset, so a step is one 32-bit addition
                constexpr uint32_t kHi = (1024u >> 4) | 1u << 14 | 2u << 29;
                constexpr uint32_t kLoS = (16u >> 4) << 16, kLoV = (kBlk >> 4) << 16;
                // (a CTA of a cluster has its rank in the bits above its shared-memory offsets)
                const uint32_t off0 = base & 0x3ffffu;
                const uint32_t q_lo = ((off0 + L::Q + (PAIR ? hh * L::TILE : 0)) >> 4) | kLoS;
                const uint32_t ts = tmem + hh * 128, to = tmem + 256 + hh * 128;
                auto desc = [](uint32_t lo) { return (uint64_t)kHi << 32 | lo; };
                uint64_t *q_full = &bars[kQFull + (PAIR ? hh : 0)], *q_empty = &bars[kQEmpty + (PAIR ? hh : 0)];
                // PAIR: the K stages and the V stages, both chains'.  ALT: the chain's one
                // ring in both roles
                struct Ring {
                    uint64_t *full, *empty;
                    uint32_t addr, phase;
                    int st, n;
                    YOCO_DEV void advance() {
                        if (++st == n) {
                            st = 0;
                            phase ^= 1;
                        }
                    }
                };
                const bool one = PAIR || hh == 0;
                Ring rk = {&bars[one ? kKFull : kVFull], &bars[one ? kKEmpty : kVEmpty], (off0 + (one ? L::K : L::V)) >> 4, 0,
                           0, L::KST};
                Ring rv_own = {&bars[kVFull], &bars[kVEmpty], (off0 + L::V) >> 4, 0, 0, L::VST};
                Ring &rv = PAIR ? rv_own : rk;
                bool ok = true;
                int seg = 0;
                uint32_t g = 0, k = 0, turn = 0;   // the chain's tiles, segments and turns
                for (; ok && !*abort_flag && it.next(p, sg); ++seg) {
                    const int nt = sg.t1 - sg.t0;
                    // tiles of this chain and of chain B; the node tile, if this chain has it
                    const int mine = PAIR ? nt : (nt + 1 - hh) / 2, others_b = PAIR ? nt : nt / 2;
                    const int n_ctx = sg.n_ctx_tiles - sg.t0;
                    const int n_nodes = PAIR ? n_ctx : (n_ctx & 1) == hh ? n_ctx >> 1 : -1;
                    ok = wait1(q_full, seg & 1);
                    if (!ok) break;
                    if (mine == 0) {   // nothing for this chain, which has its say on Q all the same
                        mbar_arrive(q_empty);
                        continue;
                    }
                    // step n: P V of tile n - 1 and S of tile n, the chains in turns (A's step
                    // 0, B's step 0, A's step 1, ...), so that one chain's MMAs run under the
                    // other's softmax: unordered, the two fall into step, with the exponentials
                    // of both at once and then the MMAs of both at once
                    for (int n = 0; n <= mine; ++n) {
                        uint32_t vd = 0;
                        uint64_t *v_empty = nullptr;
                        if (n > 0) {
                            ok = wait1(&rv.full[rv.st], rv.phase) &&
                                 (!PAIR || hh == 0 || wait1(&bars[kVClean + rv.st], rv.phase)) &&
                                 (n > 1 || k == 0 || wait1(&bars[kOFree + hh], (k - 1) & 1));
                            vd = (rv.addr + rv.st * (L::TILE >> 4)) | kLoV;
                            v_empty = &rv.empty[rv.st];
                            rv.advance();
                        }
                        ok = ok && (n == mine || wait1(&rk.full[rk.st], rk.phase));
                        if (hh == 1 || (others_b > 0 && n > 0)) ok = ok && wait1(&bars[kTurn + hh], turn++ & 1);
                        if (n > 0) ok = ok && wait1(&bars[kPHalf + hh], g & 1);
                        if (!ok) break;
                        tc::fence_after_sync();
                        if (n > 0) {
                            // the first 64 keys while the softmax forms the weights of the others
                            tc::mma_bf16_ts(to, ts, desc(vd), idPV, n > 1 ? 1u : 0u);
#pragma unroll
                            for (int kk = 1; kk < kTreeMaxNodes / 16; ++kk)
                                tc::mma_bf16_ts(to, ts + kk * 8, desc(vd + kk * (2048 >> 4)), idPV, 1u);
                            ok = wait1(&bars[kPFull + hh], g++ & 1);
                            if (!ok) break;
                            tc::fence_after_sync();
                            if (n - 1 != n_nodes) {
#pragma unroll
                                for (int kk = kTreeMaxNodes / 16; kk < BN / 16; ++kk)
                                    tc::mma_bf16_ts(to, ts + kk * 8, desc(vd + kk * (2048 >> 4)), idPV, 1u);
                            }
                            tc::mma_commit(v_empty);
                        }
                        if (n < mine) {
                            const uint32_t kd = (rk.addr + rk.st * (L::TILE >> 4)) | kLoS;
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = ((kk >> 2) * kBlk + (kk & 3) * 32) >> 4;
                                tc::mma_bf16_ss(ts, desc(q_lo + off), desc(kd + off), idS, kk > 0 ? 1u : 0u);
                            }
                        }
                        if (hh == 1 || n <= others_b - (others_b == 0)) mbar_arrive(&bars[kTurn + (hh ^ 1)]);
                        if (n < mine) {
                            tc::mma_commit(&bars[kSFull + hh]);
                            tc::mma_commit(&rk.empty[rk.st]);
                            rk.advance();
                            if (n == mine - 1) tc::mma_commit(q_empty);
                        }
                        if (n > 0) tc::mma_commit(&bars[kODone + hh]);
                    }
                    if (!ok) break;
                    // as many of chain B's turns behind chain A as it has steps
                    if (hh == 0 && others_b == mine) ok = wait1(&bars[kTurn], turn++ & 1);
                    ++k;
                }
                if (!ok) *abort_flag = 1;
                // every MMA issued by this thread has finished before TMEM is freed
                tc::mma_commit(&bars[kDrain + hh]);
                wait1(&bars[kDrain + hh], 0);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        Iter it = segments();
        Seg sg;
        const int hh = warp >> 2;
        const int r = threadIdx.x & 127;           // row in tile == TMEM lane
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + hh * 128 + lane_off;
        const uint32_t tO = tmem + 256 + hh * 128 + lane_off;
        const uint64_t sl2 = tc::f2_pack(p.scale_log2, p.scale_log2);
        float2 *s_ml = reinterpret_cast<float2 *>(sbase + L::ML);
        const bool o_32B = (reinterpret_cast<uintptr_t>(p.o) & 31u) == 0;
        bool ok = true;
        int u = 0, seg = 0, g[2] = {0, 0}, k[2] = {0, 0};   // tiles, segments, and each chain's
        for (; ok && it.next(p, sg); ++seg) {
            const int nt = sg.t1 - sg.t0;
            const int row = sg.rt * RS + (PAIR ? hh * 128 : 0) + r;   // of the stream's KV head
            const int node = row >> p.lg;
            const bool live = node < sg.n;
            const bool active = __any_sync(0xffffffffu, live);        // some row of the warp
            // stored positions of this chain's next ring tile, slot 128 t + lane + 32 e in
            // next_sp[e]: loaded a tile ahead
            int next_sp[4] = {-1, -1, -1, -1};
            auto load_slots = [&](int t) {
                if (RING && t < min(sg.t1, sg.n_ctx_tiles)) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = t * BN + lane + 32 * e;
                        next_sp[e] = j < sg.ctx ? p.slot_pos[sg.row0 + j] : -1;
                    }
                }
            };
            load_slots(sg.t0 + (PAIR ? 0 : hh));

            // what this row sees; the nodes only matter to the segment with their tile
            const bool with_nodes = sg.t1 > sg.n_ctx_tiles;
            uint64_t vis = 0;
            if (with_nodes && live) vis = p.mask ? p.mask[(int64_t)sg.b * p.N + node] : (2ull << node) - 1;
            RingBounds rb = {-1, -1};
            RingSpan span;
            if constexpr (RING) {
                // lane j has nodes j and j + 32
                const int64_t *np = p.node_pos + (int64_t)sg.b * p.N;
                const int64_t p0 = lane < sg.n ? np[lane] : 0, p1 = lane + 32 < sg.n ? np[lane + 32] : 0;
                RingBounds x0 = ring_bounds(p0, p.window), x1 = ring_bounds(p1, p.window);
                const bool e0 = lane < sg.n, e1 = lane + 32 < sg.n;
                span.any.lo = __reduce_min_sync(0xffffffffu, min(e0 ? x0.lo : INT32_MAX, e1 ? x1.lo : INT32_MAX));
                span.every.lo = __reduce_max_sync(0xffffffffu, max(e0 ? x0.lo : -1, e1 ? x1.lo : -1));
                span.every.hi = __reduce_min_sync(0xffffffffu, min(e0 ? x0.hi : INT32_MAX, e1 ? x1.hi : INT32_MAX));
                span.any.hi = __reduce_max_sync(0xffffffffu, max(e0 ? x0.hi : -1, e1 ? x1.hi : -1));
                if (active) {
                    const int src = node & 31;
                    const int lo0 = __shfl_sync(0xffffffffu, x0.lo, src), hi0 = __shfl_sync(0xffffffffu, x0.hi, src);
                    const int lo1 = __shfl_sync(0xffffffffu, x1.lo, src), hi1 = __shfl_sync(0xffffffffu, x1.hi, src);
                    if (live) rb = node < 32 ? RingBounds{lo0, hi0} : RingBounds{lo1, hi1};
                    if (with_nodes) {
                        // node by node of the warp's rows: which nodes lie in its window, a
                        // ballot of the lanes' two
#pragma unroll 4
                        for (int i = 0; i < 32 >> p.lg; ++i) {
                            const int at = __shfl_sync(0xffffffffu, node, i << p.lg) & 63;
                            const int64_t m0 = __shfl_sync(0xffffffffu, p0, at & 31), m1 = __shfl_sync(0xffffffffu, p1, at & 31);
                            const int64_t mine = at < 32 ? m0 : m1;
                            const uint32_t w0 = __ballot_sync(0xffffffffu, in_window(mine, p0, p.window));
                            const uint32_t w1 = __ballot_sync(0xffffffffu, in_window(mine, p1, p.window));
                            if (lane >> p.lg == i) vis &= (uint64_t)w1 << 32 | w0;
                        }
                    }
                }
            }
            if (sg.n < 64) vis &= (1ull << sg.n) - 1;

            float m = -INFINITY, l = 0.f;
            bool first = true;
            for (int t = sg.t0; t < sg.t1; ++t, ++u) {
                if (!PAIR && hh != ((t - sg.t0) & 1)) {
                    ++g[hh ^ 1];
                    continue;
                }
                const bool nodes = t == sg.n_ctx_tiles;
                const int j0 = t * BN;
                // is the tile seen whole by every row?
                bool masked = nodes || j0 + BN > sg.ctx;
                int sp[4];
                if constexpr (RING) {
                    if (!nodes) {
                        bool all = true;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sp[e] = next_sp[e];
                            all &= span.every.hi > span.every.lo && span.every.sees(sp[e]);
                        }
                        masked = !__all_sync(0xffffffffu, all);
                    }
                    load_slots(t + (PAIR ? 1 : 2));
                }
                if (!waitw(&bars[kSFull + hh], g[hh] & 1)) { ok = false; break; }
                tc::fence_after_sync();
                if (masked && (!PAIR || hh == 0)) {
                    // V rows before P V: thread r has key row r.  After S of this tile,
                    // which was issued after the stage's last tenant had landed, so the
                    // parity below cannot mean an older phase
                    const int at = PAIR ? u : 2 * g[hh] + 1;   // copies before it in its ring
                    const int vst = PAIR || hh == 1 ? L::VST : L::KST, v0 = PAIR || hh == 1 ? kVFull : kKFull;
                    if (!waitw(&bars[v0 + at % vst], (at / vst) & 1)) { ok = false; break; }
                    uint8_t *tile = sbase + (PAIR || hh == 1 ? L::V : L::K) + (at % vst) * L::TILE;
                    bool odd = false;
                    if (nodes) {
                        // 64 rows, two threads a row
                        odd = clean_v_row<KB, 4>(tile, r & 63, (r >> 6) * 4, (r & 63) >= sg.n);
                    } else if (RING) {
                        int s = -1;
#pragma unroll
                        for (int e = 0; e < 4; ++e) s = (warp & 3) == e ? sp[e] : s;
                        if (!(span.every.hi > span.every.lo && span.every.sees(s)))
                            odd = clean_v_row<KB, 8>(tile, r, 0, !(span.any.hi > span.any.lo && span.any.sees(s)));
                    } else if (j0 + r >= sg.ctx) {
                        clean_v_row<KB, 8>(tile, r, 0, true);
                    }
                    if (odd) *(volatile int *)&misc->poison[seg & 7] = seg;
                    fence_proxy_async_smem();
                }
                if (active) {
                    float s[BN];
#pragma unroll
                    for (int c = 0; c < BN; c += 32) tc::tmem_ld32(tS + c, s + c);
                    tc::wait_ld();
                    if (masked) {
                        uint32_t w[4];
                        if (nodes) {
                            w[0] = (uint32_t)vis;
                            w[1] = (uint32_t)(vis >> 32);
                            w[2] = w[3] = 0;
                        } else if constexpr (RING) {
                            // node by node of the warp's rows: a ballot is the node's word
#pragma unroll 4
                            for (int i = 0; i < 32 >> p.lg; ++i) {
                                const RingBounds x = {__shfl_sync(0xffffffffu, rb.lo, i << p.lg),
                                                      __shfl_sync(0xffffffffu, rb.hi, i << p.lg)};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t word = __ballot_sync(0xffffffffu, x.sees(sp[e]));
                                    if (lane >> p.lg == i) w[e] = word;
                                }
                            }
                        } else {
                            const int cnt = sg.ctx - j0;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int x = cnt - 32 * e;
                                w[e] = x >= 32 ? 0xffffffffu : x <= 0 ? 0u : (1u << x) - 1u;
                            }
                        }
                        // most masked tiles are masked in one chunk of 32 columns
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!__all_sync(0xffffffffu, w[e] == 0xffffffffu)) {
#pragma unroll
                                for (int c = 0; c < 32; ++c) s[32 * e + c] = w[e] >> c & 1u ? s[32 * e + c] : -INFINITY;
                            }
                    }
                    float a8[8];
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) a8[kk] = max3_nan(s[kk], s[kk + 8], s[kk + 16]);
#pragma unroll
                    for (int c = 24; c < 120; c += 16)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) a8[kk] = max3_nan(a8[kk], s[c + kk], s[c + 8 + kk]);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) a8[kk] = max3_nan(a8[kk], a8[kk], s[120 + kk]);
                    const float mx = max3_nan(max3_nan(a8[0], a8[1], a8[2]), max3_nan(a8[3], a8[4], a8[5]),
                                              max3_nan(a8[6], a8[6], a8[7]));
                    // the reference moves (and O is rescaled) only when it grows by more than
                    // 2^8; a NaN or +inf score makes it NaN, and with it the row
                    const float m_cand = mx * p.scale_log2;
                    float alpha = 1.f;
                    const bool grow = m_cand > m + 8.f;
                    if (grow) {
                        alpha = m == -INFINITY ? 0.f : tc::ex2(m - m_cand);
                        m = m_cand;
                    }
                    if (!(mx < INFINITY)) m = NAN;
                    const float neg_m = m == -INFINITY ? 0.f : -m;
                    const uint64_t nm2 = tc::f2_pack(neg_m, neg_m);
                    if (!first && __any_sync(0xffffffffu, grow)) {
                        if (!waitw(&bars[kODone + hh], (g[hh] - 1) & 1)) { ok = false; break; }
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tc::tmem_ld32(tO + c, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= alpha;
                            tc::tmem_st32(tO + c, o);
                        }
                    }
                    uint64_t rs2a = 0, rs2b = 0;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t pk[BN / 4];
#pragma unroll
                        for (int cc = 0; cc < BN / 2; cc += 2) {
                            const int c = half * (BN / 2) + cc;
                            float x0, x1;
                            tc::f2_unpack(tc::f2_fma(tc::f2_pack(s[c], s[c + 1]), sl2, nm2), x0, x1);
                            const float e0 = tc::ex2(x0), e1 = tc::ex2(x1);
                            if (c & 2)
                                rs2b = tc::f2_add(rs2b, tc::f2_pack(e0, e1));
                            else
                                rs2a = tc::f2_add(rs2a, tc::f2_pack(e0, e1));
                            // P is rounded to bf16 for the tensor core (half a step of each
                            // weight); the sum takes the weights before that
                            pk[cc / 2] = tc::pack_bf16x2(e0, e1);
                        }
                        tc::tmem_st32u(tS + half * 32, pk);
                        if (half == 0) {
                            tc::wait_st();
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars[kPHalf + hh]);
                        }
                    }
                    float ra0, ra1, rb0, rb1;
                    tc::f2_unpack(rs2a, ra0, ra1);
                    tc::f2_unpack(rs2b, rb0, rb1);
                    l = l * alpha + ((ra0 + ra1) + (rb0 + rb1));
                    tc::wait_st();
                } else {
                    __syncwarp();   // the rows of V that it has cleaned
                    if (lane == 0) mbar_arrive(&bars[kPHalf + hh]);
                }
                first = false;
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars[kPFull + hh]);
                    if (PAIR && hh == 0) mbar_arrive(&bars[kVClean + u % L::VST]);   // chain B's P V reads this tile too
                }
                ++g[hh];
            }
            if (!ok) break;
            const bool has_b = PAIR || nt >= 2;
            if (!PAIR && hh == 1) {
                // chain B leaves its statistics for chain A, which joins and writes both
                if (has_b) {
                    if (k[1] >= 1 && !waitw(&bars[kOFree + 1], (k[1] - 1) & 1)) { ok = false; break; }
                    s_ml[r] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[kML]);
                }
                ++k[0];
                k[1] += has_b;
                continue;
            }
            if (!waitw(&bars[kODone + hh], (g[hh] - 1) & 1)) { ok = false; break; }
            if constexpr (CLUSTER && PAIR) {
                // The partial goes over the tiles in shared memory, which the other chain's P V may
                // still be reading.  A parity alone does not tell its last P V from the one two
                // before.  Chain B therefore tells chain A that it has seen its own finish.  For
                // chain B the parity will do: its last P V was issued behind chain A's last one,
                // that behind chain A's last S, which was read by then, and an S finishes after the
                // P V before it.
                if (hh == 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[kML]);
                    if (!waitw(&bars[kODone], (g[hh] - 1) & 1)) { ok = false; break; }
                } else if (!waitw(&bars[kML], k[1] & 1)) {
                    ok = false;
                    break;
                }
            }
            float wa = 1.f, wb = 0.f;
            const bool join = !PAIR && has_b;
            if (join) {
                if (!waitw(&bars[kML], k[1] & 1) || !waitw(&bars[kODone + 1], (g[1] - 1) & 1)) { ok = false; break; }
                const float2 ml = s_ml[r];
                const float mm = fmaxf(m, ml.x);
                const float ref = mm == -INFINITY ? 0.f : mm;
                wa = tc::ex2(m - ref);
                wb = tc::ex2(ml.x - ref);
                l = l * wa + ml.y * wb;
                m = mm;
            }
            tc::fence_after_sync();
            const bool poison = *(volatile int *)&misc->poison[seg & 7] == seg;
            const bool none = m == -INFINITY && l == 0.f;   // a NaN sum is not nothing
            const float inv = none ? 0.f : 1.f / l;
            const int head = (sg.g << p.lg) + (row & ((1 << p.lg) - 1));
            const int64_t entry = (int64_t)blockIdx.x * 2 + sg.slot;
            const int ws_row = (PAIR ? hh * 128 : 0) + r;
            __nv_bfloat16 *dst =
                static_cast<__nv_bfloat16 *>(p.o) + (((int64_t)sg.b * p.N + (live ? node : 0)) * p.Hq + head) * D;
            if (active) {
#pragma unroll 2
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tc::tmem_ld32(tO + c, o);
                    if (join) {
                        float ob[32];
                        tc::tmem_ld32(tO + 128 + c, ob);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = o[e] * wa + ob[e] * wb;
                    } else {
                        tc::wait_ld();
                    }
                    if (poison && live) {
                        const __nv_bfloat16 *vn = static_cast<const __nv_bfloat16 *>(p.v_nodes) +
                                                  ((int64_t)sg.b * p.N * p.Hkv + sg.g) * D + c;
                        if (sg.t1 > sg.n_ctx_tiles)
                            for (int j = 0; j < sg.n; ++j)
                                if ((vis >> j) & 1) add_odd(vn + (int64_t)j * p.Hkv * D, o);
                        if constexpr (RING) {
                            const int j1 = min(sg.t1 * BN, sg.ctx);
                            for (int j = sg.t0 * BN; j < j1; ++j)
                                if (rb.sees(p.slot_pos[sg.row0 + j]))
                                    add_odd(static_cast<const __nv_bfloat16 *>(p.v) +
                                                ((sg.row0 + j) * p.Hkv + sg.g) * D + c, o);
                        }
                    }
                    if (CLUSTER) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(sbase + ((uint32_t)ws_row * (D + 4) + c + e) * 4) =
                                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    } else if (live && sg.whole) {
                        // 32-byte stores where o allows them: a thread's row is its own, so a
                        // warp's store covers 32 rows, and these are whole sectors
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            uint32_t wv[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) wv[u] = tc::pack_bf16x2(o[e + 2 * u] * inv, o[e + 2 * u + 1] * inv);
                            if (o_32B) {
                                st_global_32B(dst + c + e, wv);
                            } else {
                                *reinterpret_cast<uint4 *>(dst + c + e) = make_uint4(wv[0], wv[1], wv[2], wv[3]);
                                *reinterpret_cast<uint4 *>(dst + c + e + 8) = make_uint4(wv[4], wv[5], wv[6], wv[7]);
                            }
                        }
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            p.ws_o[(entry * (D / 4) + (c + e) / 4) * RS + ws_row] =
                                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                    __syncwarp();   // the TMEM load takes the whole warp
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[kOFree + hh]);
                if (join) mbar_arrive(&bars[kOFree + 1]);
            }
            if (CLUSTER) reinterpret_cast<float2 *>(sbase + RS * (D + 4) * 4)[ws_row] = make_float2(m, l);
            if (!CLUSTER && live && sg.whole && p.lse)
                p.lse[((int64_t)sg.b * p.Hq + head) * p.N + node] = none ? -INFINITY : (m + __log2f(l)) * kLn2;
            if (!CLUSTER && live && !sg.whole) p.ws_ml[entry * RS + ws_row] = make_float2(m, l);
            ++k[0];
            k[1] += has_b;
        }
        // a CTA without a tile, and one that gave up: nothing to add
        if (CLUSTER && (seg == 0 || !ok) && (PAIR || hh == 0))
            reinterpret_cast<float2 *>(sbase + RS * (D + 4) * 4)[(PAIR ? hh * 128 : 0) + r] = make_float2(-INFINITY, 0.f);
        if (!ok) *abort_flag = 1;
        tc::wait_st();   // no TMEM store may be in flight when TMEM is freed
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
    if constexpr (CLUSTER) {
        // Join the partials of the cluster's CTAs: every warp of every CTA has rows of
        // its own, and reads them from all of them.  Rows without a node come out as
        // zeros.  Every CTA gets here whatever happened before: its waits are bounded.
        __syncwarp();
        clu::sync_all();
        const Seg &s = misc->share.s;
        const int P = p.cluster, rank = (int)clu::rank();
        const int rows = min(RS, (p.N << p.lg) - s.rt * RS);
        const uint32_t ml0 = base + RS * (D + 4) * 4;
        for (int i = warp * P + rank; i < rows; i += P * (kThreads / 32)) {
            const int row = s.rt * RS + i, node = row >> p.lg, head = (s.g << p.lg) + (row & ((1 << p.lg) - 1));
            float m = -INFINITY, l = 0.f;
            if (node < s.n && lane < P) {
                const uint32_t at = clu::map_rank(ml0 + i * 8, lane);
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(m), "=f"(l) : "r"(at) : "memory");
            }
            const bool some = !(m == -INFINITY && l == 0.f);
            const uint32_t parts = __ballot_sync(0xffffffffu, some);
            const float mm = warp_max(m), ref = mm == -INFINITY ? 0.f : mm;
            const float w = some ? tc::ex2(m - ref) : 0.f;
            const float sum = warp_sum(w * l);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int j = 0; j < P; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j);
                if (!((parts >> j) & 1) || lane >= D / 4) continue;
                float4 o;
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(o.x), "=f"(o.y), "=f"(o.z), "=f"(o.w)
                             : "r"(clu::map_rank(base + ((uint32_t)i * (D + 4) + 4 * lane) * 4, j))
                             : "memory");
                acc.x = fmaf(wj, o.x, acc.x);
                acc.y = fmaf(wj, o.y, acc.y);
                acc.z = fmaf(wj, o.z, acc.z);
                acc.w = fmaf(wj, o.w, acc.w);
            }
            const float inv = parts ? 1.f / sum : 0.f;
            if (lane < D / 4) {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.o) + (((int64_t)s.b * p.N + node) * p.Hq + head) * D;
                *reinterpret_cast<uint2 *>(dst + 4 * lane) =
                    make_uint2(tc::pack_bf16x2(acc.x * inv, acc.y * inv), tc::pack_bf16x2(acc.z * inv, acc.w * inv));
            }
            if (p.lse && lane == 0)
                p.lse[((int64_t)s.b * p.Hq + head) * p.N + node] = parts ? (mm + __log2f(sum)) * kLn2 : -INFINITY;
        }
        __syncwarp();
        clu::sync_all();   // no CTA leaves while another reads its shared memory
    }
}

// ------------------------------------------------------------------- host
namespace {

// 4-D bf16 map over [d3, d2, d1, D] (innermost D), 128-byte swizzle.
bool make_map(CUtensorMap *m, const void *ptr, int64_t D, int64_t d1, int64_t d2, int64_t d3, int box1, int box2) {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)d1, (uint64_t)d2, (uint64_t)d3};
    const uint64_t row = (uint64_t)(d1 * D * 2);
    // an extent of one has no stride of its own
    const uint64_t strides[3] = {(uint64_t)(D * 2), row, d3 > 1 ? (uint64_t)d2 * row : row};
    const uint32_t box[4] = {64, (uint32_t)box1, (uint32_t)box2, 1};
    return encode_bf16_map_4d(m, ptr, dims, strides, box);
}

template <typename F>
bool has_registers(F *kern) {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess && a.numRegs >= kRegs;
}

template <int D, bool RING, bool PAIR>
cudaError_t launch_tc(const TreeArgs &a, const TreePlan &pl, cudaStream_t st) {
    const int G = a.Hq / a.Hkv;
    CUtensorMap mq, mk, mv, mkn, mvn;
    const int64_t ctx_rows = RING ? a.window : a.cache_rows, ctx_b = RING ? a.B : 1;
    if (!make_map(&mq, a.q, D, a.Hq, a.N, a.B, G, 128 / G) || !make_map(&mk, a.k, D, a.Hkv, ctx_rows, ctx_b, 1, BN) ||
        !make_map(&mv, a.v, D, a.Hkv, ctx_rows, ctx_b, 1, BN) ||
        !make_map(&mkn, a.k_nodes, D, a.Hkv, a.N, a.B, 1, kTreeMaxNodes) ||
        !make_map(&mvn, a.v_nodes, D, a.Hkv, a.N, a.B, 1, kTreeMaxNodes))
        return cudaErrorNotSupported;
    constexpr size_t smem = Smem<D, PAIR>::ALLOC;
    const bool cl = pl.cluster > 0;
    auto kern = cl ? tree_tc_kernel<D, RING, PAIR, true> : tree_tc_kernel<D, RING, PAIR, false>;
    // a build with fewer registers than kRegs would wait for the rest for good
    static const bool regs_ok[2] = {has_registers(tree_tc_kernel<D, RING, PAIR, false>),
                                    has_registers(tree_tc_kernel<D, RING, PAIR, true>)};
    if (!regs_ok[cl]) return cudaErrorInvalidDeviceFunction;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    note_launches(1);
    if (!cl)
        return launch_pdl(kern, dim3(pl.heads * pl.groups), dim3(kThreads), smem, st, mq, mk, mv, mkn, mvn,
                          make_params(a, pl));
    const int n_rt = (a.N * G + pl.rows - 1) / pl.rows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * n_rt * a.Hkv * pl.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)pl.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, mkn, mvn, make_params(a, pl));
}

template <int D>
cudaError_t launch_tc_d(const TreeArgs &a, const TreePlan &pl, cudaStream_t st) {
    const bool pair = pl.rows == 256;
    if (a.window > 0) return pair ? launch_tc<D, true, true>(a, pl, st) : launch_tc<D, true, false>(a, pl, st);
    return pair ? launch_tc<D, false, true>(a, pl, st) : launch_tc<D, false, false>(a, pl, st);
}

}  // namespace
}  // namespace tree

cudaError_t launch_tree_tc(const TreeArgs &a, const TreePlan &pl, cudaStream_t st) {
    if (a.D == 128) return tree::launch_tc_d<128>(a, pl, st);
    if (a.D == 64) return tree::launch_tc_d<64>(a, pl, st);
    return cudaErrorNotSupported;
}

unsigned int read_and_clear_status_tree_tc() {
    unsigned int h = 0, z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_tree_tc, sizeof(h)) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_status_tree_tc, &z, sizeof(z));
    return h;
}

}  // namespace yoco
