// Attention of drafted tokens over the shared cache or the self-decoder's ring
// (sm_100a): the work plan, the CUDA-core kernel and the join of shared
// streams.
//
// A decoder that drafts several tokens ahead checks them in one pass: node i of
// a tree of up to 64 drafted tokens attends to the sequence's context and to
// its own ancestors among the nodes.  The cross-decoder's context is the one
// shared cache ("YOCO: Caching Once for Decoder-Decoder Long-Context Language
// Models", podcast transcript, cue 26), the self-decoder's the window ring
// ("You Only Cache Once", paperlayer summary, section 3 "Sliding-Window
// Attention"); the pages do not draft.  With x_j = scale q k_j over the keys
// that a row sees, m = max x, l = sum e^(x_j - m): o = sum e^(x_j - m) v_j / l,
// lse = m + ln l, and o = 0, lse = -inf for a row that sees nothing.
#include "tree.cuh"

#include <algorithm>
#include <type_traits>

namespace yoco {

static __device__ unsigned int g_status_tree;

namespace tree {
namespace {

constexpr int kFewThreads = 512, kRowThreads = 256;
constexpr int kFewStages = 3;
constexpr int kSimtKeys = 64;   // BN of the CUDA-core kernels
constexpr int kMergeWarps = 8;
constexpr int kGroupHeads = 8;
// tiles of a CTA of a cluster at most, by whether the clusters fill half the GPU
// (16 nodes, 16 tiles a CTA: 2 x 8059 tokens in clusters on 64 SMs 23.4 us, as
// shares 21.9; 4 x 8059, on 128 SMs, 29.6 and 35.0; 12 tiles a CTA: 2 x 6011
// tokens 19.6 and 19.8)
constexpr int kClusterTiles = 16, kFewClusterTiles = 12;

// A tile of the fp32 kernels: where its keys are, and how many there are.
struct Tile {
    const float *k, *v;
    int64_t row0;
    int cnt, j0;
    bool nodes;
};
YOCO_DEV Tile tile_of(const Params &p, const Seg &g, int t) {
    Tile x;
    x.nodes = t == g.n_ctx_tiles;
    x.j0 = x.nodes ? 0 : t * kSimtKeys;
    x.cnt = x.nodes ? g.n : min(kSimtKeys, g.ctx - x.j0);
    x.row0 = x.nodes ? (int64_t)g.b * p.N : g.row0 + x.j0;
    x.k = static_cast<const float *>(x.nodes ? p.k_nodes : p.k);
    x.v = static_cast<const float *>(x.nodes ? p.v_nodes : p.v);
    return x;
}

// Shared memory of a CTA: stages of K and V rows, PITCH floats apart, and of a
// ring's stored positions.
template <int PITCH>
struct Stage {
    static constexpr int FLOATS = 2 * kSimtKeys * PITCH;
    float *k, *v;
    int *slot;
    YOCO_DEV Stage(float *base, int *slots, int i)
        : k(base + i * FLOATS), v(k + kSimtKeys * PITCH), slot(slots + i * kSimtKeys) {}
};

// Starts the copy of a tile's K, V or both into a stage (rows past its keys as zeros).
template <int D, bool RING, int THREADS, int PITCH, bool K, bool V>
YOCO_DEV void load_tile(const Params &p, const Seg &g, int t, const Stage<PITCH> &s) {
    const Tile x = tile_of(p, g, t);
    for (int c = threadIdx.x; c < kSimtKeys * (D / 4); c += THREADS) {
        const int j = c / (D / 4), d = (c % (D / 4)) * 4;
        const bool there = j < x.cnt;
        const int64_t off = there ? ((x.row0 + j) * p.Hkv + g.g) * D + d : 0;
        const uint32_t bytes = there ? 16 : 0;
        if (K)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(s.k + j * PITCH + d)),
                         "l"(x.k + off), "r"(bytes) : "memory");
        if (V)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(s.v + j * PITCH + d)),
                         "l"(x.v + off), "r"(bytes) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (RING && K && !x.nodes && threadIdx.x < kSimtKeys)
        s.slot[threadIdx.x] = threadIdx.x < x.cnt ? p.slot_pos[x.row0 + threadIdx.x] : -1;
}

// The rows of a row block: Q (scaled) into shared memory, what they see.
template <int D, bool RING, int RS, int THREADS, int PITCH>
YOCO_DEV void load_rows(const Params &p, const Seg &g, int rows, float *sq, uint64_t *s_nodes, RingBounds *s_bounds) {
    const int G = 1 << p.lg;
    for (int c = threadIdx.x; c < RS * (D / 4); c += THREADS) {
        const int r = c / (D / 4), d = (c % (D / 4)) * 4, rr = g.rt * RS + r;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows)
            x = *reinterpret_cast<const float4 *>(
                static_cast<const float *>(p.q) +
                (((int64_t)g.b * p.N + (rr >> p.lg)) * p.Hq + (g.g << p.lg) + (rr & (G - 1))) * D + d);
        *reinterpret_cast<float4 *>(sq + r * PITCH + d) =
            make_float4(x.x * p.scale_log2, x.y * p.scale_log2, x.z * p.scale_log2, x.w * p.scale_log2);
    }
    if (threadIdx.x < RS) {
        const int i = (g.rt * RS + (int)threadIdx.x) >> p.lg;
        const bool there = (int)threadIdx.x < rows;
        s_nodes[threadIdx.x] = there ? visible_nodes<RING>(p, g.b, g.n, i) : 0;
        if (RING)
            s_bounds[threadIdx.x] =
                there ? ring_bounds(p.node_pos[(int64_t)g.b * p.N + i], p.window) : RingBounds{-1, -1};
    }
}

// A finished row: to o and lse, or as a partial.
template <int D, int RS>
YOCO_DEV void store_four(const Params &p, const Seg &g, int r, int col4, float m, float L, float4 o) {
    const int rr = g.rt * RS + r, node = rr >> p.lg, h = (g.g << p.lg) + (rr & ((1 << p.lg) - 1));
    if (g.whole) {
        const bool none = m == -INFINITY && L == 0.f;   // a NaN sum is not nothing
        const float inv = none ? 0.f : 1.f / L;
        float *dst = static_cast<float *>(p.o) + (((int64_t)g.b * p.N + node) * p.Hq + h) * D;
        *reinterpret_cast<float4 *>(dst + 4 * col4) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (p.lse && col4 == 0)
            p.lse[((int64_t)g.b * p.Hq + h) * p.N + node] = none ? -INFINITY : (m + log2f(L)) * kLn2;
    } else {
        const int64_t e = (int64_t)blockIdx.x * 2 + g.slot;
        if (col4 == 0) p.ws_ml[e * RS + r] = make_float2(m, L);
        p.ws_o[(e * (D / 4) + col4) * RS + r] = o;
    }
}

}  // namespace

// fp32 on the CUDA cores, up to 32 rows of a KV head: instructions bound it more
// than anything else does (69% of the issue slots are taken, 40-45% of the FMA
// pipe, 34-55% of DRAM; two tiles are on their way while one computes).  A warp
// has eight rows and KW keys of every tile, with statistics of its own, so that
// nothing is exchanged before the segment ends.  A lane has CPL
// columns of q, K, V and o: K and V are read from shared memory once, in whole
// rows, and q stays in registers.  The columns' sums for four keys by eight rows
// are exchanged so that a lane ends with one of the 32 scores; its q and K are
// loaded in an order that puts what it keeps first, so that no exchange has to
// choose.  A key that a row does not see is left out of the product (its weight is
// held as -1), so what its K and V hold never reaches the row.
// Over 8 x 8192 keys of 8 heads, D = 128: 8 rows take 118 us (4.5 TB/s), 16 take
// 192, 32 take 317 (390 in the kernel below).  With a lane per key and q in shared
// memory, where an operand that all lanes share costs as much as one that they do
// not, 138, 221 and 368; with exchanges that choose, the same; with pairs of rows in
// packed FMAs 155, 265 and 462.
template <int D, bool RING, int RS>
__global__ void __launch_bounds__(kFewThreads, 1) tree_few_kernel(const __grid_constant__ Params p) {
    constexpr int BN = kSimtKeys, PITCH = D, CPL = D / 32, WARPS = kFewThreads / 32;
    constexpr int RG = RS / 8, KG = WARPS / RG, KW = BN / KG;
    using Cols = std::conditional_t<CPL == 4, float4, float2>;
    union Lane {
        Cols all;
        float c[CPL];
    };
    extern __shared__ __align__(16) float smem[];
    __shared__ Range s_range;
    __shared__ uint64_t s_nodes[RS];
    __shared__ RingBounds s_bounds[RS];
    __shared__ int s_slot[kFewStages * BN];
    __shared__ float2 s_ml[WARPS][8];
    __shared__ __align__(16) float s_w[WARPS][4][8];
    float *sq = smem;
    float *const stages = sq + RS * PITCH;
    float *const red = stages;   // [warp][8 rows][D] when the segment ends
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x < 32) find_range<RING, RS, BN>(p, &s_range);
    __syncthreads();
    fill_rows_without_node<float, D, RING, RS, BN>(p, threadIdx.x / 32, WARPS, &g_status_tree);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kg = warp / RG, rq = warp % RG * 8;
    const int row = rq + (lane >> 2);   // of this lane's score
    SegIter<RING, RS, BN> it(p, s_range);
    Seg g;
    while (it.next(p, g)) {
        const int rows = min(RS, (g.n << p.lg) - g.rt * RS);
        for (int i = 0; i < kFewStages - 1; ++i) {
            if (g.t0 + i < g.t1)
                load_tile<D, RING, kFewThreads, PITCH, true, true>(p, g, g.t0 + i, Stage<PITCH>(stages, s_slot, i));
            else asm volatile("cp.async.commit_group;" ::: "memory");
        }
        load_rows<D, RING, RS, kFewThreads, PITCH>(p, g, rows, sq, s_nodes, s_bounds);
        __syncthreads();
        float m = -INFINITY, l = 0.f;
        float o[8][CPL];
        Lane q[8];   // of row r ^ lane / 4
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            q[r].all = *reinterpret_cast<const Cols *>(sq + (rq + (r ^ lane >> 2)) * PITCH + lane * CPL);
#pragma unroll
            for (int c = 0; c < CPL; ++c) o[r][c] = 0.f;
        }
        for (int t = g.t0, st = 0; t < g.t1; ++t, st = st + 1 == kFewStages ? 0 : st + 1) {
            const Stage<PITCH> cur(stages, s_slot, st);
            asm volatile("cp.async.wait_group %0;" ::"n"(kFewStages - 2) : "memory");
            __syncthreads();   // this tile is here; the one before is no longer read
            if (t + kFewStages - 1 < g.t1)
                load_tile<D, RING, kFewThreads, PITCH, true, true>(p, g, t + kFewStages - 1,
                                                Stage<PITCH>(stages, s_slot, st == 0 ? kFewStages - 1 : st - 1));
            else asm volatile("cp.async.commit_group;" ::: "memory");
            const Tile x = tile_of(p, g, t);
#pragma unroll 1
            for (int k0 = kg * KW; k0 < min((kg + 1) * KW, x.cnt); k0 += 4) {
                float s[32];   // [row ^ lane / 4][key ^ lane % 4]
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    Lane kk;
                    kk.all = *reinterpret_cast<const Cols *>(cur.k + (k0 + (k ^ (lane & 3))) * PITCH + lane * CPL);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        s[4 * r + k] = q[r].c[0] * kk.c[0];
#pragma unroll
                        for (int c = 1; c < CPL; ++c) s[4 * r + k] = fmaf(q[r].c[c], kk.c[c], s[4 * r + k]);
                    }
                }
#pragma unroll
                for (int n = 16; n > 0; n >>= 1)
#pragma unroll
                    for (int i = 0; i < n; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i + n], n);
                const float score = s[0];
                const int key = k0 + (lane & 3);
                const bool see = x.nodes ? (s_nodes[row] >> key) & 1
                                 : RING  ? key < x.cnt && s_bounds[row].sees(cur.slot[key])
                                         : key < x.cnt;
                const bool all = __all_sync(0xffffffffu, see);
                // a new maximum: rare after the first tiles (a NaN score is none, and
                // reaches the row by its exponential)
                if (__any_sync(0xffffffffu, see && score > m)) {
                    float mx = see ? fmaxf(m, score) : m;
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float al = mx == -INFINITY ? 1.f : exp2f(m - mx);
                    m = mx;
                    l *= al;
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float f = __shfl_sync(0xffffffffu, al, 4 * r);
#pragma unroll
                        for (int c = 0; c < CPL; ++c) o[r][c] *= f;
                    }
                }
                const float e = exp2f(score - (m == -INFINITY ? 0.f : m));
                if (see) l += e;
                __syncwarp();   // the last weights are read
                s_w[warp][lane & 3][lane >> 2] = see ? e : -1.f;
                __syncwarp();
                if (all) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        Lane v;
                        v.all = *reinterpret_cast<const Cols *>(cur.v + (k0 + k) * PITCH + lane * CPL);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float4 y = *reinterpret_cast<const float4 *>(&s_w[warp][k][4 * h]);
                            const float w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                            for (int r = 0; r < 4; ++r)
#pragma unroll
                                for (int c = 0; c < CPL; ++c) o[4 * h + r][c] = fmaf(w[r], v.c[c], o[4 * h + r][c]);
                        }
                    }
                } else {
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        Lane v;
                        v.all = *reinterpret_cast<const Cols *>(cur.v + (k0 + k) * PITCH + lane * CPL);
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const float w = s_w[warp][k][r];
                            if (!(w < 0.f))   // seen (a NaN is)
#pragma unroll
                                for (int c = 0; c < CPL; ++c) o[r][c] = fmaf(w, v.c[c], o[r][c]);
                        }
                    }
                }
            }
        }
        __syncthreads();   // before the stages are used for the join
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if ((lane & 3) == 0) s_ml[warp][lane >> 2] = make_float2(m, l);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            Lane x;
#pragma unroll
            for (int c = 0; c < CPL; ++c) x.c[c] = o[r][c];
            *reinterpret_cast<Cols *>(red + (warp * 8 + r) * D + lane * CPL) = x.all;
        }
        __syncthreads();
        for (int r = warp; r < rows && lane < D / 4; r += WARPS) {   // the KG key groups of a row
            float M = -INFINITY, L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < KG; ++k) M = fmaxf(M, s_ml[k * RG + r / 8][r % 8].x);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int k = 0; k < KG; ++k) {
                const int from = k * RG + r / 8;
                const float2 ml = s_ml[from][r % 8];
                const float w = exp2f(ml.x - ref);
                const float4 y = *reinterpret_cast<const float4 *>(red + (from * 8 + r % 8) * D + 4 * lane);
                L = fmaf(w, ml.y, L);
                acc.x = fmaf(w, y.x, acc.x);
                acc.y = fmaf(w, y.y, acc.y);
                acc.z = fmaf(w, y.z, acc.z);
                acc.w = fmaf(w, y.w, acc.w);
            }
            store_four<D, RS>(p, g, r, lane, M, L, acc);
        }
        __syncthreads();   // before the next segment's first tiles
    }
}

// fp32 on the CUDA cores, more rows: operands are read from shared memory for
// every few FMAs, and no unit is full (69% of the issue slots, 57% of the FMA
// pipe).  256 threads for 16 RT rows x 64 keys; thread (ty, tx) of a
// 16 x 16 grid holds the rows ty + 16 i: in S = q K^T the keys tx + 16 j, in O += P V
// the columns 4 tx + 64 j.  V is copied while S is computed, the next K during P V.
// A row's statistics are the same in its 16 threads; unseen keys as in the kernel
// above.  64 nodes, G = 4, over 8 x 4096 keys: 932 us in blocks of 128 rows (37
// TFLOP/s), 1052 in blocks of 64; 24 nodes 524 and about 600.
template <int D, bool RING, int RT>
__global__ void __launch_bounds__(kRowThreads, 1) tree_simt_kernel(const __grid_constant__ Params p) {
    constexpr int RS = 16 * RT, BN = kSimtKeys, NJ = D / 64;
    constexpr int PITCH = D + 4, PP = BN + 16;   // eight keys, and two rows, on different banks
    extern __shared__ __align__(16) float smem[];
    __shared__ Range s_range;
    __shared__ uint64_t s_nodes[RS];
    __shared__ RingBounds s_bounds[RS];
    __shared__ int s_slot[BN];
    float *sq = smem, *sp = sq + RS * PITCH;
    const Stage<PITCH> cur(sp + RS * PP, s_slot, 0);
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x < 32) find_range<RING, RS, BN>(p, &s_range);
    __syncthreads();
    fill_rows_without_node<float, D, RING, RS, BN>(p, threadIdx.x / 32, kRowThreads / 32, &g_status_tree);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    SegIter<RING, RS, BN> it(p, s_range);
    Seg g;
    while (it.next(p, g)) {
        const int rows = min(RS, (g.n << p.lg) - g.rt * RS);
        load_tile<D, RING, kRowThreads, PITCH, true, false>(p, g, g.t0, cur);
        load_rows<D, RING, RS, kRowThreads, PITCH>(p, g, rows, sq, s_nodes, s_bounds);
        float m[RT], l[RT], o[RT][NJ * 4];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < NJ * 4; ++e) o[i][e] = 0.f;
        }
        for (int t = g.t0; t < g.t1; ++t) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();   // K is here; the V before is no longer read
            load_tile<D, RING, kRowThreads, PITCH, false, true>(p, g, t, cur);
            const Tile x = tile_of(p, g, t);
            float s[RT][4] = {};
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 a[RT], bk[4];
#pragma unroll
                for (int i = 0; i < RT; ++i) a[i] = *reinterpret_cast<const float4 *>(sq + (ty + 16 * i) * PITCH + d);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    bk[j] = *reinterpret_cast<const float4 *>(cur.k + (tx + 16 * j) * PITCH + d);
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i][j] = fmaf(a[i].x, bk[j].x, s[i][j]);
                        s[i][j] = fmaf(a[i].y, bk[j].y, s[i][j]);
                        s[i][j] = fmaf(a[i].z, bk[j].z, s[i][j]);
                        s[i][j] = fmaf(a[i].w, bk[j].w, s[i][j]);
                    }
            }
            bool all = true;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                bool see[4];
                float mx = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = tx + 16 * j;
                    if (x.nodes) see[j] = (s_nodes[ty + 16 * i] >> c) & 1;
                    else if (RING) see[j] = c < x.cnt && s_bounds[ty + 16 * i].sees(cur.slot[c]);
                    else see[j] = c < x.cnt;
                    all &= see[j];
                    // a NaN score has to reach the row: fmaxf would drop it, the exponential below does not
                    if (see[j]) mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                const float al = mx == -INFINITY ? 1.f : exp2f(m[i] - mx);
                const float ref = mx == -INFINITY ? 0.f : mx;
                m[i] = mx;
                l[i] *= al;
#pragma unroll
                for (int e = 0; e < NJ * 4; ++e) o[i][e] *= al;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = exp2f(s[i][j] - ref);
                    if (see[j]) l[i] += e;
                    sp[(ty + 16 * i) * PP + tx + 16 * j] = see[j] ? e : -1.f;
                }
            }
            all = __all_sync(0xffffffffu, all);
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();   // V is here; K is no longer read
            if (t + 1 < g.t1) load_tile<D, RING, kRowThreads, PITCH, true, false>(p, g, t + 1, cur);
            if (all) {
#pragma unroll 2
                for (int c = 0; c < BN; c += 4) {
                    float w[RT][4];
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const float4 y = *reinterpret_cast<const float4 *>(sp + (ty + 16 * i) * PP + c);
                        w[i][0] = y.x, w[i][1] = y.y, w[i][2] = y.z, w[i][3] = y.w;
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            const float4 v =
                                *reinterpret_cast<const float4 *>(cur.v + (c + u) * PITCH + 4 * tx + 64 * j);
#pragma unroll
                            for (int i = 0; i < RT; ++i) {
                                o[i][4 * j] = fmaf(w[i][u], v.x, o[i][4 * j]);
                                o[i][4 * j + 1] = fmaf(w[i][u], v.y, o[i][4 * j + 1]);
                                o[i][4 * j + 2] = fmaf(w[i][u], v.z, o[i][4 * j + 2]);
                                o[i][4 * j + 3] = fmaf(w[i][u], v.w, o[i][4 * j + 3]);
                            }
                        }
                }
            } else {
                for (int c = 0; c < x.cnt; ++c) {
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const float pp = sp[(ty + 16 * i) * PP + c];
                        if (pp < 0.f) continue;   // not seen (a NaN goes on)
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            const float4 v = *reinterpret_cast<const float4 *>(cur.v + c * PITCH + 4 * tx + 64 * j);
                            o[i][4 * j] = fmaf(pp, v.x, o[i][4 * j]);
                            o[i][4 * j + 1] = fmaf(pp, v.y, o[i][4 * j + 1]);
                            o[i][4 * j + 2] = fmaf(pp, v.z, o[i][4 * j + 2]);
                            o[i][4 * j + 3] = fmaf(pp, v.w, o[i][4 * j + 3]);
                        }
                    }
                }
            }
        }
        __syncthreads();   // before the next segment is loaded
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            float L = l[i];
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) L += __shfl_xor_sync(0xffffffffu, L, w);
            if (ty + 16 * i >= rows) continue;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                store_four<D, RS>(p, g, ty + 16 * i, tx + 16 * j, m[i], L,
                                  make_float4(o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]));
        }
    }
}

// Joins the partials of shared streams.  A lane has one row, a warp 32 rows'
// four columns at a time (COLS of those groups of four, a group apart from the
// next warp's): partials are stored by column, so its loads are whole.  grid.x:
// a block of 32 rows, and of columns; grid.y: a candidate stream of a head block
// -- every stream, or, where there are more streams than shares, the one that
// share grid.y + 1 starts inside of (the first of its shares to do so); grid.z:
// the head in its block.
template <typename T, int D, bool RING, int RS, int BN, int COLS>
__global__ void __launch_bounds__(32 * kMergeWarps)
    tree_merge_kernel(const __grid_constant__ Params p, const int by_stream) {
    constexpr int GROUPS = D / 4, AHEAD = 4, COL_BLOCKS = GROUPS / (COLS * kMergeWarps);
    const int lane = threadIdx.x & 31;
    const int sub = (int)blockIdx.x % COL_BLOCKS * COLS * kMergeWarps + (threadIdx.x >> 5);   // the first group
    const int r = (int)blockIdx.x / COL_BLOCKS * 32 + lane, blocks = p.Hkv / p.heads;
    pdl_trigger();
    pdl_wait();
    const int T_all = p.prefix[p.B], part = p.prefix[p.B + 1];
    const Deal d(T_all, max(1, min(T_all, p.groups)));
    int b, stream = 0, x = 0;
    if (by_stream) {
        const int per_b = ((p.N << p.lg) + RS - 1) / RS * blocks;
        b = (int)blockIdx.y / per_b;
        stream = (int)blockIdx.y - b * per_b;
    } else {
        const int c = (int)blockIdx.y + 1;
        x = part > 0 ? c * part : c < min(T_all, p.groups) ? d.start(c) : T_all;
        if (x >= T_all) return;
        // the sequence with tile x: the last one that starts at or before it and has tiles
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (p.prefix[mid] <= x) lo = mid;
            else hi = mid;
        }
        b = lo;
    }
    const int base = p.prefix[b];
    const Seq s = sequence<RING, RS, BN>(p, b);
    const int nt = s.n_ctx_tiles + 1, numbered = s.numbered(part);
    if (!by_stream) stream = (x - base) / numbered;
    if (stream >= s.streams(p)) return;
    const int a = base + stream * numbered;
    const int c0 = part > 0 ? a / part : d.owner(a), c1 = part > 0 ? (a + nt - 1) / part : d.owner(a + nt - 1);
    if (c0 == c1 || (!by_stream && c0 != (int)blockIdx.y)) return;   // finished by its CTA; another share's
    // the stream's part in c0 opens c0's share only when it starts there
    const int first = part > 0 || d.start(c0) == a ? 0 : 1, n_part = c1 - c0 + 1;
    const int g = stream % blocks * p.heads + (int)blockIdx.z, rr = stream / blocks * RS + r;
    const int node = rr >> p.lg, h = (g << p.lg) + (rr & ((1 << p.lg) - 1));
    if (r >= RS || node >= s.n) return;
    float M = -INFINITY, L = 0.f;
    float4 acc[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n_part; i0 += AHEAD) {
        float2 ml[AHEAD];
        float4 o[AHEAD][COLS];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int c = 0; c < COLS; ++c) o[u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + u < n_part) {
                const int64_t e = (int64_t)((c0 + i0 + u) * p.heads + (int)blockIdx.z) * 2 + (i0 + u == 0 ? first : 0);
                ml[u] = p.ws_ml[e * RS + r];
#pragma unroll
                for (int c = 0; c < COLS; ++c) o[u][c] = p.ws_o[(e * GROUPS + sub + c * kMergeWarps) * RS + r];
            }
        }
        float mx = M;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) mx = fmaxf(mx, ml[u].x);
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float keep = exp2f(M - ref);
        L *= keep;
#pragma unroll
        for (int c = 0; c < COLS; ++c)
            acc[c] = make_float4(acc[c].x * keep, acc[c].y * keep, acc[c].z * keep, acc[c].w * keep);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const float w = exp2f(ml[u].x - ref);
            L = fmaf(w, ml[u].y, L);
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                acc[c].x = fmaf(w, o[u][c].x, acc[c].x);
                acc[c].y = fmaf(w, o[u][c].y, acc[c].y);
                acc[c].z = fmaf(w, o[u][c].z, acc[c].z);
                acc[c].w = fmaf(w, o[u][c].w, acc[c].w);
            }
        }
        M = mx;
    }
    const bool none = M == -INFINITY && L == 0.f;
    const float inv = none ? 0.f : 1.f / L;
    T *dst = static_cast<T *>(p.o) + (((int64_t)b * p.N + node) * p.Hq + h) * D;
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
        T v[4] = {from_f32<T>(acc[c].x * inv), from_f32<T>(acc[c].y * inv), from_f32<T>(acc[c].z * inv),
                  from_f32<T>(acc[c].w * inv)};
        using Out = std::conditional_t<sizeof(T) == 2, uint2, uint4>;
        *reinterpret_cast<Out *>(dst + 4 * (sub + c * kMergeWarps)) = *reinterpret_cast<Out *>(v);
    }
    if (p.lse && sub == 0)
        p.lse[((int64_t)b * p.Hq + h) * p.N + node] = none ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ------------------------------------------------------------------- host
namespace {

template <int D, bool RING>
cudaError_t launch_fp32(const TreeArgs &a, const TreePlan &pl, cudaStream_t st) {
    const bool few = pl.rows <= 32;
    const size_t smem = sizeof(float) * (few ? pl.rows * D + kFewStages * Stage<D>::FLOATS
                                             : pl.rows * (D + 4 + kSimtKeys + 16) + Stage<D + 4>::FLOATS);
    auto kern = pl.rows == 8    ? tree_few_kernel<D, RING, 8>
                : pl.rows == 16 ? tree_few_kernel<D, RING, 16>
                : pl.rows == 32 ? tree_few_kernel<D, RING, 32>
                : pl.rows == 64 ? tree_simt_kernel<D, RING, 4>
                                : tree_simt_kernel<D, RING, 8>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    note_launches(1);
    return launch_pdl(kern, dim3(pl.heads * pl.groups), dim3(few ? kFewThreads : kRowThreads), smem, st,
                      make_params(a, pl));
}

template <typename T, int D, bool RING, int RS, int BN>
cudaError_t launch_merge(const TreeArgs &a, const TreePlan &pl, cudaStream_t st) {
    const int rows = std::min(RS, a.N * (a.Hq / a.Hkv));
    const int64_t streams = (int64_t)a.B * ((a.N * (a.Hq / a.Hkv) + RS - 1) / RS) * (a.Hkv / pl.heads);
    const bool by_stream = streams <= pl.groups - 1;
    const int most = by_stream ? (int)streams : pl.groups - 1;   // shared streams of a head
    if (most == 0) return cudaSuccess;                           // one share: nothing to join
    // enough blocks of rows to fill the GPU: every column to one CTA; else spread
    constexpr int ALL = D / 4 / kMergeWarps;
    const int row_blocks = (rows + 31) / 32;
    const bool whole = (int64_t)row_blocks * most * pl.heads >= 2 * device_sm_count();
    note_launches(1);
    return launch_pdl(whole ? tree_merge_kernel<T, D, RING, RS, BN, ALL> : tree_merge_kernel<T, D, RING, RS, BN, 1>,
                      dim3((unsigned)(row_blocks * (whole ? 1 : ALL)), (unsigned)most, (unsigned)pl.heads),
                      dim3(32 * kMergeWarps), 0, st, make_params(a, pl), (int)by_stream);
}

template <int D, bool RING>
cudaError_t launch_d(const TreeArgs &a, const TreePlan &pl, cudaStream_t st) {
    if (a.dtype == kBF16) {
        const cudaError_t e = launch_tree_tc(a, pl, st);
        if (e != cudaSuccess || pl.cluster) return e;
        return pl.rows == 128 ? launch_merge<__nv_bfloat16, D, RING, 128, kTcKeys>(a, pl, st)
                              : launch_merge<__nv_bfloat16, D, RING, 256, kTcKeys>(a, pl, st);
    }
    const cudaError_t e = launch_fp32<D, RING>(a, pl, st);
    if (e != cudaSuccess) return e;
    switch (pl.rows) {
        case 8: return launch_merge<float, D, RING, 8, kSimtKeys>(a, pl, st);
        case 16: return launch_merge<float, D, RING, 16, kSimtKeys>(a, pl, st);
        case 32: return launch_merge<float, D, RING, 32, kSimtKeys>(a, pl, st);
        case 64: return launch_merge<float, D, RING, 64, kSimtKeys>(a, pl, st);
        default: return launch_merge<float, D, RING, 128, kSimtKeys>(a, pl, st);
    }
}

}  // namespace
}  // namespace tree

bool make_tree_plan(int32_t B, int32_t N, int64_t max_len, int Hq, int Hkv, int D, int dtype, TreePlan *plan) {
    TreePlan pl;
    // the 16-byte chunks of a token's heads (up to 32 each) and the rows are counted in 32 bits
    if (Hq > 1 << 24 || (int64_t)B * N > (int64_t)INT32_MAX / 2 / Hq) return false;
    // bf16: the tensor-core kernel, one row tile of 128 or two; fp32: CUDA cores, in
    // row blocks of 8, 16, 32, 64 or 128 (what they take: at the kernels)
    const int R = N * (Hq / Hkv);
    pl.rows = dtype == kBF16 ? R <= 128 ? 128 : 256 : R <= 8 ? 8 : R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128;
    pl.keys = dtype != kBF16 ? tree::kSimtKeys : tree::kTcKeys;
    const int n_rt = (N * (Hq / Hkv) + pl.rows - 1) / pl.rows;
    const int64_t stream_tiles = (max_len + pl.keys - 1) / pl.keys + 1;
    // bf16, few streams, none of them long: a cluster a stream, no second launch
    // and no numbering to work out first (16 nodes over 1 x 1915 tokens 10.4 us,
    // as shares 16.8; over 4 x 3963 17.2 and 20.9; over 8 x 3963 30.0 and 34.7).
    // All clusters have to run at once -- 16 clusters of eight took two rounds
    // and lost to the shares -- and the 148 SMs' partitions hold 15 of eight CTAs
    // this big, 33 of four and 74 of two.  The limits on tiles are safe ones for one
    // row tile.  What they give away: two row tiles lose from about six tiles a CTA
    // on unless the clusters fill half the GPU (64 nodes over 2 x 6011 tokens 35.7 us
    // in clusters, 27.4 as shares), and one row tile would gain past the limits (16
    // nodes over 1 x 15227 tokens 23.1 and 24.5, over 4 x 12155 39.6 and 44.7; two
    // streams of 15227 tokens 22.1 and 31.1).
    const int sms = device_sm_count(), room[3] = {sms / 2, (sms - 16) / 4, (sms - 28) / 8};
    pl.cluster = 0;
    if (dtype == kBF16)
        for (int i = 0; i < 3; ++i)
            if (const int64_t streams = (int64_t)B * n_rt * Hkv, c = 2 << i;
                streams <= room[i] &&
                stream_tiles <= c * (streams * c * 2 >= sms ? tree::kClusterTiles : tree::kFewClusterTiles))
                pl.cluster = (int)c;
    if (pl.cluster) {
        pl.heads = pl.groups = 1;
        pl.ml_off = pl.o_off = pl.ws_bytes = 0;
        *plan = pl;
        return true;
    }
    // groups of CTAs, one KV head of a block each (tree.cuh): the largest divisor of Hkv up to 8
    pl.heads = 1;
    for (int h = 2; h <= tree::kGroupHeads; ++h)
        if (Hkv % h == 0) pl.heads = h;
    // tiles at full length: no group without a tile is launched
    const int64_t blocks = (int64_t)B * n_rt * (Hkv / pl.heads);
    const int64_t tiles = blocks * stream_tiles;
    if (tiles > INT32_MAX / 2) return false;
    pl.groups = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, sms / pl.heads));
    pl.ml_off = ((size_t)(B + 2) * sizeof(int32_t) + 15) / 16 * 16;
    const size_t entries = (size_t)pl.groups * pl.heads * 2 * pl.rows;
    pl.o_off = pl.ml_off + entries * sizeof(float2);
    pl.ws_bytes = pl.o_off + entries * D * sizeof(float);
    *plan = pl;
    return true;
}

cudaError_t launch_tree(const TreeArgs &a, const TreePlan &pl, cudaStream_t st) {
    if (a.D == 128) return a.window > 0 ? tree::launch_d<128, true>(a, pl, st) : tree::launch_d<128, false>(a, pl, st);
    if (a.D == 64) return a.window > 0 ? tree::launch_d<64, true>(a, pl, st) : tree::launch_d<64, false>(a, pl, st);
    return cudaErrorNotSupported;
}

unsigned int read_and_clear_status_tree() {
    unsigned int h = 0, z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_tree, sizeof(h)) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_status_tree, &z, sizeof(z));
    return h;
}

}  // namespace yoco
