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

constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 32;     // RS of the CUDA-core kernel
constexpr int kSimtKeys = 64;     // BN of the CUDA-core kernel
constexpr int kMergeWarps = 8;
constexpr int kGroupHeads = 8;
// tiles of a CTA of a cluster at most, by whether the clusters fill half the GPU
// (16 nodes over 2 x 8000 tokens, 16 tiles in clusters on 64 SMs, 26.1 us, as
// shares 23.7; over 4 x 7900, on 128 SMs, 27.3 and 33.6)
constexpr int kClusterTiles = 16, kFewClusterTiles = 12;

template <typename T>
YOCO_DEV void load16(const T *src, float *f) {
    Chunk<T>::unpack(*reinterpret_cast<const uint4 *>(src), f);
}

}  // namespace

// CUDA-core kernel: 256 threads for 32 rows x 64 keys.  Thread (ty, tx) of a
// 16 x 16 grid holds rows 2 ty, 2 ty + 1: in S = q K^T the keys tx, tx + 16,
// tx + 32, tx + 48; in O += P V the columns 4 tx + 64 j.  A row's statistics
// are the same in its 16 threads.  P of a key that the row does not see is -1
// in shared memory, and the product leaves such a key out, so what its K and V
// hold (infinities, NaN) never reaches the row.
template <typename T, int D, bool RING>
__global__ void __launch_bounds__(kSimtThreads) tree_simt_kernel(const __grid_constant__ Params p) {
    constexpr int RS = kSimtRows, BN = kSimtKeys, PITCH = D + 4, PP = BN + 4;
    constexpr int EPC = Chunk<T>::N, NJ = D / 64;
    extern __shared__ __align__(16) float smem[];
    float *sq = smem, *sk = sq + RS * PITCH, *sv = sk + BN * PITCH, *sp = sv + BN * PITCH;
    __shared__ Range s_range;
    __shared__ uint64_t s_nodes[RS];
    __shared__ int s_slot[BN];
    __shared__ RingBounds s_bounds[RS];
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x < 32) find_range<RING, RS, BN>(p, &s_range);
    __syncthreads();
    fill_rows_without_node<T, D, RING, RS, BN>(p, threadIdx.x / 32, kSimtThreads / 32, &g_status_tree);
    const int G = 1 << p.lg;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    SegIter<RING, RS, BN> it(p, s_range);
    Seg g;
    while (it.next(p, g)) {
        const int rows = min(RS, g.n * G - g.rt * RS);
        __syncthreads();
        for (int c = tid; c < RS * (D / EPC); c += kSimtThreads) {
            const int r = c / (D / EPC), d = (c % (D / EPC)) * EPC;
            float f[EPC];
#pragma unroll
            for (int e = 0; e < EPC; ++e) f[e] = 0.f;
            if (r < rows) {
                const int rr = g.rt * RS + r;
                load16(static_cast<const T *>(p.q) +
                           (((int64_t)g.b * p.N + rr / G) * p.Hq + g.g * G + rr % G) * D + d, f);
            }
#pragma unroll
            for (int e = 0; e < EPC; ++e) sq[r * PITCH + d + e] = f[e] * p.scale_log2;
        }
        if (tid < RS) {
            const int i = (g.rt * RS + tid) / G;
            s_nodes[tid] = tid < rows ? visible_nodes<RING>(p, g.b, g.n, i) : 0;
            if (RING) {
                if (tid < rows) s_bounds[tid] = ring_bounds(p.node_pos[(int64_t)g.b * p.N + i], p.window);
                else s_bounds[tid] = RingBounds{-1, -1};
            }
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[2][NJ * 4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < NJ * 4; ++e) o[i][e] = 0.f;

        for (int t = g.t0; t < g.t1; ++t) {
            const bool nodes = t == g.n_ctx_tiles;
            const int j0 = nodes ? 0 : t * BN;
            const int cnt = nodes ? g.n : min(BN, g.ctx - j0);
            const int64_t row0 = nodes ? (int64_t)g.b * p.N : g.row0 + j0;
            const T *kb = static_cast<const T *>(nodes ? p.k_nodes : p.k);
            const T *vb = static_cast<const T *>(nodes ? p.v_nodes : p.v);
            __syncthreads();
            for (int c = tid; c < BN * (D / EPC); c += kSimtThreads) {
                const int j = c / (D / EPC), d = (c % (D / EPC)) * EPC;
                float fk[EPC], fv[EPC];
#pragma unroll
                for (int e = 0; e < EPC; ++e) fk[e] = fv[e] = 0.f;
                if (j < cnt) {
                    const int64_t off = ((row0 + j) * p.Hkv + g.g) * D + d;
                    load16(kb + off, fk);
                    load16(vb + off, fv);
                }
#pragma unroll
                for (int e = 0; e < EPC; e += 4) {
                    *reinterpret_cast<float4 *>(sk + j * PITCH + d + e) = make_float4(fk[e], fk[e + 1], fk[e + 2], fk[e + 3]);
                    *reinterpret_cast<float4 *>(sv + j * PITCH + d + e) = make_float4(fv[e], fv[e + 1], fv[e + 2], fv[e + 3]);
                }
            }
            if (RING && !nodes && tid < BN)
                s_slot[tid] = tid < cnt ? p.slot_pos[(int64_t)g.b * p.window + j0 + tid] : -1;
            __syncthreads();

            float s[2][4] = {};
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 a[2], bk[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) a[i] = *reinterpret_cast<const float4 *>(sq + (2 * ty + i) * PITCH + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) bk[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * PITCH + d);
#pragma unroll
                for (int i = 0; i < 2; ++i)
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
            for (int i = 0; i < 2; ++i) {
                bool see[4];
                float mx = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = tx + 16 * j;
                    if (nodes) see[j] = (s_nodes[2 * ty + i] >> c) & 1;
                    else if (RING) see[j] = c < cnt && s_bounds[2 * ty + i].sees(s_slot[c]);
                    else see[j] = c < cnt;
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
                    sp[(2 * ty + i) * PP + tx + 16 * j] = see[j] ? e : -1.f;
                }
            }
            all = __all_sync(0xffffffffu, all);
            __syncwarp();
            if (all) {
#pragma unroll 4
                for (int c = 0; c < BN; ++c) {
                    const float p0 = sp[(2 * ty) * PP + c], p1 = sp[(2 * ty + 1) * PP + c];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const float4 v = *reinterpret_cast<const float4 *>(sv + c * PITCH + 4 * tx + 64 * j);
                        o[0][4 * j] = fmaf(p0, v.x, o[0][4 * j]);
                        o[0][4 * j + 1] = fmaf(p0, v.y, o[0][4 * j + 1]);
                        o[0][4 * j + 2] = fmaf(p0, v.z, o[0][4 * j + 2]);
                        o[0][4 * j + 3] = fmaf(p0, v.w, o[0][4 * j + 3]);
                        o[1][4 * j] = fmaf(p1, v.x, o[1][4 * j]);
                        o[1][4 * j + 1] = fmaf(p1, v.y, o[1][4 * j + 1]);
                        o[1][4 * j + 2] = fmaf(p1, v.z, o[1][4 * j + 2]);
                        o[1][4 * j + 3] = fmaf(p1, v.w, o[1][4 * j + 3]);
                    }
                }
            } else {
                for (int c = 0; c < cnt; ++c) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float pp = sp[(2 * ty + i) * PP + c];
                        if (pp < 0.f) continue;   // not seen (a NaN goes on)
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            const float4 v = *reinterpret_cast<const float4 *>(sv + c * PITCH + 4 * tx + 64 * j);
                            o[i][4 * j] = fmaf(pp, v.x, o[i][4 * j]);
                            o[i][4 * j + 1] = fmaf(pp, v.y, o[i][4 * j + 1]);
                            o[i][4 * j + 2] = fmaf(pp, v.z, o[i][4 * j + 2]);
                            o[i][4 * j + 3] = fmaf(pp, v.w, o[i][4 * j + 3]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float L = l[i];
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) L += __shfl_xor_sync(0xffffffffu, L, w);
            const int r = 2 * ty + i;
            if (r >= rows) continue;
            const int rr = g.rt * RS + r, node = rr / G, h = g.g * G + rr % G;
            if (g.whole) {
                const bool none = m[i] == -INFINITY && L == 0.f;   // a NaN sum is not nothing
                const float inv = none ? 0.f : 1.f / L;
                T *dst = static_cast<T *>(p.o) + (((int64_t)g.b * p.N + node) * p.Hq + h) * D;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[4 * tx + 64 * j + e] = from_f32<T>(o[i][4 * j + e] * inv);
                if (p.lse && tx == 0)
                    p.lse[((int64_t)g.b * p.Hq + h) * p.N + node] =
                        none ? -INFINITY : (m[i] + log2f(L)) * kLn2;
            } else {
                const int64_t e = (int64_t)blockIdx.x * 2 + g.slot;
                if (tx == 0) p.ws_ml[e * RS + r] = make_float2(m[i], L);
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    p.ws_o[(e * (D / 4) + tx + 16 * j) * RS + r] =
                        make_float4(o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]);
            }
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
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const __grid_constant__ Params p, const int by_stream) {
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

template <typename T, int D, bool RING>
cudaError_t launch_simt(const TreeArgs &a, const TreePlan &pl, cudaStream_t st) {
    constexpr size_t smem = sizeof(float) * ((kSimtRows + 2 * kSimtKeys) * (D + 4) + kSimtRows * (kSimtKeys + 4));
    auto kern = tree_simt_kernel<T, D, RING>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    note_launches(1);
    return launch_pdl(kern, dim3(pl.heads * pl.groups), dim3(kSimtThreads), smem, st, make_params(a, pl));
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
    const cudaError_t e = launch_simt<float, D, RING>(a, pl, st);
    if (e != cudaSuccess) return e;
    return launch_merge<float, D, RING, kSimtRows, kSimtKeys>(a, pl, st);
}

}  // namespace
}  // namespace tree

bool make_tree_plan(int32_t B, int32_t N, int64_t max_len, int Hq, int Hkv, int D, int dtype, TreePlan *plan) {
    TreePlan pl;
    // bf16: the tensor-core kernel, one row tile of 128 or two; fp32: CUDA cores
    pl.rows = dtype != kBF16 ? tree::kSimtRows : N * (Hq / Hkv) <= 128 ? 128 : 256;
    pl.keys = dtype != kBF16 ? tree::kSimtKeys : tree::kTcKeys;
    const int n_rt = (N * (Hq / Hkv) + pl.rows - 1) / pl.rows;
    const int64_t stream_tiles = (max_len + pl.keys - 1) / pl.keys + 1;
    // bf16, few streams, none of them long: a cluster a stream, no second launch
    // and no numbering to work out first (16 nodes over 1 x 2047 tokens 12.3 us,
    // as shares 19.3; over 8 x 3900 28.0 and 38.5; over 1 x 15000 25.4 and 26.5).
    // All clusters have to run at once -- 16 clusters of eight took two rounds
    // and lost to the shares -- and the GPU's partitions hold 15 of eight CTAs this
    // big, 33 of four and 74 of two.
    const int sms = device_sm_count(), room[3] = {sms / 2, (sms - 16) / 4, (sms - 28) / 8};
    pl.cluster = 0;
    if (dtype == kBF16)
        for (int i = 0; i < 3; ++i)
            if (const int64_t streams = (int64_t)B * n_rt * Hkv, c = 2 << i;
                streams <= room[i] && stream_tiles <= c * (streams * c * 2 >= sms ? tree::kClusterTiles : tree::kFewClusterTiles))
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
    if ((int64_t)B * N * Hq > (int64_t)INT32_MAX / 2 || tiles > INT32_MAX / 2) return false;
    const int64_t ctas = (int64_t)(dtype != kBF16 ? 2 : 1) * sms;
    pl.groups = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, ctas / pl.heads));
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
