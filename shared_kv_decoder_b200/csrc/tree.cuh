// What the tree-decode kernels share: their parameters, how the work is dealt
// to the CTAs, and which keys a drafted token sees.
//
// Work.  A "stream" is the rows of one (sequence, row block, KV head): RS rows
// of the row order r = node * G + head-in-group (G = Hq / Hkv), against that
// sequence's keys in tiles of BN -- first the context (the cache's rows, or the
// ring's slots), then one tile with the drafted nodes' own keys.  The CTAs come
// in groups of `heads`, one KV head each, which walk the same tiles side by
// side: a token's K (or V) of all heads is one run in memory.  It matters where
// the keys come from DRAM and segments are short (8 heads of 128, 64 sequences x
// 48 nodes over the 1024 ring, caches flushed: 121 us, 127 in groups of one; with
// the ring in L2 119 and 118), and no more over long contexts (64 nodes over
// 131007 tokens 160 and 158, 16 sequences of 64K-128K tokens 976-1047 and 990-996).
// The tiles of (sequence, row block, head block) are numbered sequence by
// sequence, and group c of C takes a contiguous share of the T tiles, T / C of
// them to within one: every CTA gets the same work whatever the lengths are,
// and a long stream is shared by as many CTAs as it has work for.  Where a few
// more tiles a group (kAlignSlack) let every stream be cut into parts of `part`
// tiles with no group holding pieces of two, it is cut so: a second segment
// costs a CTA another fill and drain of its pipeline, as long as about five
// tiles (16 nodes over the 1024 ring, 12 sequences: 21 us, cut anywhere 27; 16
// sequences: 22 and 35; on the other side 12 x 8000 tokens, 81 and 78).  The
// streams are then numbered as if they were a multiple of `part` long.  A CTA's part of a stream
// is a segment.  A stream that one CTA has whole is finished by it; of one that
// is shared, each CTA leaves a partial (m, l, unnormalised o) in the workspace,
// slot 0 for the segment its share opens with, slot 1 for the one it ends with,
// and tree_merge_kernel joins them.
//
// Few streams, none of them long, are not numbered: a cluster of CTAs has each,
// and its CTAs join their parts through each other's shared memory (tree.cu says
// when, tree_tc.cu how).
#pragma once

#include "common.cuh"
#include "launch.h"
#include "schedule.h"

namespace yoco {
namespace tree {

constexpr int kTcKeys = 128;   // keys of a tile of the tensor-core kernel

struct Params {
    const void *q, *k_nodes, *v_nodes;   // [B, N, Hq, D], [B, N, Hkv, D]
    const void *k, *v;                   // cache [cache_rows, Hkv, D] or ring [B, window, Hkv, D]
    const int64_t *seq_start;            // cache only
    const int32_t *seq_len;
    const int32_t *slot_pos;             // ring only
    const int64_t *node_pos;
    const uint64_t *mask;                // [B, N] or null (a chain)
    const int32_t *n_nodes;              // [B] or null (N each)
    int32_t B, N, Hq, Hkv;
    int32_t lg;                          // log2 of Hq / Hkv
    int32_t heads, groups;               // KV heads of a CTA group; groups
    int32_t cluster;                     // CTAs of a cluster, 0: no clusters
    int32_t window;                      // 0: cache
    int64_t cache_rows, max_len;
    float scale_log2;
    void *o;                             // [B, N, Hq, D]
    float *lse;                          // [B, Hq, N] or null
    int32_t *prefix;                     // workspace: first tile of each sequence, the total, the part
    float2 *ws_ml;                       // workspace: [2 grid][RS]
    float4 *ws_o;                        // workspace: [2 grid][D / 4][RS], a row's four columns each
};

// One sequence: its nodes (0 when it has none or is out of range), context
// keys, context tiles and row blocks.
struct Seq {
    int n, n_ctx_tiles, n_rt;
    int ctx;
    int64_t row0;
    bool ok;
    YOCO_DEV int streams(const Params &p) const { return n_rt * (p.Hkv / p.heads); }
    // tiles of a stream as numbered
    YOCO_DEV int numbered(int part) const {
        const int nt = n_ctx_tiles + 1;
        return part > 0 ? (nt + part - 1) / part * part : nt;
    }
};

template <bool RING, int RS, int BN>
YOCO_DEV Seq sequence(const Params &p, int b) {
    Seq s;
    const int n = p.n_nodes ? p.n_nodes[b] : p.N;
    s.ok = n >= 0 && n <= p.N;
    if (RING) {
        s.ctx = p.window;
        s.row0 = (int64_t)b * p.window;
    } else {
        s.ctx = p.seq_len[b];
        s.row0 = p.seq_start[b];
        // an empty context is in range wherever it starts inside the cache
        s.ok = s.ok && (s.ctx == 0 ? s.row0 >= 0 && s.row0 <= p.cache_rows
                                   : sched::decode_seq_ok(s.row0, s.ctx, p.max_len, p.cache_rows));
    }
    s.n = s.ok ? n : 0;
    s.n_ctx_tiles = s.ok ? (int)(((unsigned)s.ctx + BN - 1) / BN) : 0;
    s.n_rt = (int)(((unsigned)(s.n << p.lg) + RS - 1) / RS);
    return s;
}

// Shares of T tiles for C groups, C <= T: the first T mod C get one more.
struct Deal {
    int q, rem;
    YOCO_DEV Deal(int T, int C) : q(T / C), rem(T - q * C) {}
    YOCO_DEV int start(int c) const { return c * q + min(c, rem); }
    YOCO_DEV int owner(int x) const {
        const int cut = rem * (q + 1);
        return x < cut ? x / (q + 1) : rem + (x - cut) / q;
    }
};

// Where a CTA's share starts: numbered tiles [x, end), the sequence that holds
// x and that sequence's first tile.  Run by one whole warp into shared memory;
// CTA 0 also leaves the numbering in the workspace for the merge.
struct Range {
    int x, end, base, b, part;
    Seq s;
};

constexpr int kAlignSlack = 5;

template <bool RING, int RS, int BN>
YOCO_DEV void find_range(const Params &p, Range *out) {
    const int lane = threadIdx.x & 31;
    const Seq none = {};
    const Seq s0 = lane < p.B ? sequence<RING, RS, BN>(p, lane) : none;
    const int m0 = s0.streams(p);
    int T = m0 * (s0.n_ctx_tiles + 1);
    for (int b = lane + 32; b < p.B; b += 32) {
        const Seq s = sequence<RING, RS, BN>(p, b);
        T += s.streams(p) * (s.n_ctx_tiles + 1);
    }
    T = __reduce_add_sync(0xffffffffu, T);
    const int C = min(T, p.groups), c = (int)blockIdx.x / p.heads;
    int part = 0;
    if (p.B <= 32 && T > 0 && __reduce_add_sync(0xffffffffu, m0) <= C) {
        const int least = (T + C - 1) / C;
        for (int u = least; u <= least + kAlignSlack && part == 0; ++u)
            if (__reduce_add_sync(0xffffffffu, m0 * ((s0.n_ctx_tiles + u) / u)) <= C) part = u;
    }
    int x = 0, end = 0;
    bool found = T == 0;
    if (part > 0) {
        T = part * __reduce_add_sync(0xffffffffu, m0 * ((s0.n_ctx_tiles + part) / part));
        x = min(c * part, T);
        end = min(x + part, T);
    } else if (c < C) {
        const Deal d(T, C);
        x = d.start(c);
        end = d.start(c + 1);
    }
    found = x >= end;
    if (lane == 0) {
        out->x = x;
        out->end = end;
        out->part = part;
    }
    int base = 0;
    for (int b0 = 0; b0 < p.B && (!found || blockIdx.x == 0); b0 += 32) {
        const int b = b0 + lane;
        const Seq s = b0 == 0 ? s0 : b < p.B ? sequence<RING, RS, BN>(p, b) : none;
        const int cnt = s.streams(p) * s.numbered(part);
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, base + incl > x);
        if (!found && hit) {
            if (lane == __ffs(hit) - 1) {
                out->b = b;
                out->base = base + incl - cnt;
                out->s = s;
            }
            found = true;
        }
        if (blockIdx.x == 0 && b < p.B) p.prefix[b] = base + incl - cnt;
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (blockIdx.x == 0 && lane == 0) {
        p.prefix[p.B] = T;
        p.prefix[p.B + 1] = part;
    }
}

// A segment: tiles [t0, t1) of one stream.
struct Seg {
    int b, rt, g;        // sequence, row block, KV head
    int n, n_ctx_tiles;  // its nodes and context tiles (tile n_ctx_tiles holds the nodes)
    int t0, t1;
    int ctx;
    int64_t row0;
    bool whole;          // the CTA has the whole stream
    int slot;            // partial slot otherwise
};

// Steps through a CTA's segments.  Every role of a kernel runs its own copy.
template <bool RING, int RS, int BN>
struct SegIter {
    Range r;
    int x0, numbered, tiles;   // of a stream, of the sequence
    YOCO_DEV SegIter(const Params &p, const Range &range) : r(range), x0(range.x), numbered(0), tiles(0) {
        if (r.x < r.end) count(p);
    }
    YOCO_DEV void count(const Params &p) {
        numbered = r.s.numbered(r.part);
        tiles = r.s.streams(p) * numbered;
    }
    YOCO_DEV bool next(const Params &p, Seg &g) {
        if (r.x >= r.end) return false;
        while (r.x >= r.base + tiles) {
            r.base += tiles;
            r.s = sequence<RING, RS, BN>(p, ++r.b);
            count(p);
        }
        const int nt = r.s.n_ctx_tiles + 1, blocks = p.Hkv / p.heads;
        const int off = r.x - r.base, stream = off / numbered;
        g.b = r.b;
        g.rt = stream / blocks;
        g.g = (stream - g.rt * blocks) * p.heads + (int)blockIdx.x % p.heads;
        g.n = r.s.n;
        g.n_ctx_tiles = r.s.n_ctx_tiles;
        g.ctx = r.s.ctx;
        g.row0 = r.s.row0;
        g.t0 = off - stream * numbered;
        const int len = min(numbered - g.t0, r.end - r.x);
        g.t1 = min(nt, g.t0 + len);
        g.whole = g.t0 == 0 && g.t1 == nt;
        g.slot = r.x == x0 ? 0 : 1;
        r.x += len;
        return true;
    }
};

// The one segment of a CTA of a cluster: cluster c has stream c (sequence by
// sequence, row blocks outermost, at their full number), and its CTAs an equal
// share of the stream's tiles each.
struct ClusterIter {
    Seg s;
    bool any;
    YOCO_DEV bool next(const Params &, Seg &g) {
        if (!any) return false;
        any = false;
        g = s;
        return true;
    }
};

template <bool RING, int RS, int BN>
YOCO_DEV ClusterIter cluster_share(const Params &p, int cluster, int rank, int size, Seq *seq) {
    ClusterIter it;
    const int n_rt = ((p.N << p.lg) + RS - 1) / RS, per_b = n_rt * p.Hkv;
    it.s.b = cluster / per_b;
    const int stream = cluster - it.s.b * per_b;
    it.s.rt = stream / p.Hkv;
    it.s.g = stream - it.s.rt * p.Hkv;
    const Seq q = sequence<RING, RS, BN>(p, it.s.b);
    const int nt = it.s.rt < q.n_rt ? q.n_ctx_tiles + 1 : 0;
    it.s.n = q.n;
    it.s.n_ctx_tiles = q.n_ctx_tiles;
    it.s.ctx = q.ctx;
    it.s.row0 = q.row0;
    it.s.t0 = (int)((unsigned)(rank * nt) / (unsigned)size);
    it.s.t1 = (int)((unsigned)((rank + 1) * nt) / (unsigned)size);
    it.s.whole = false;
    it.s.slot = 0;
    it.any = it.s.t0 < it.s.t1;
    *seq = q;
    return it;
}

// Rows without a node, and every row of a sequence out of range (which is
// reported as bit 1 of *status): o = 0, lse = -inf.  Warp w of `warps` of every
// CTA takes its share of the (sequence, node) pairs.
constexpr unsigned int kStatusBadSequence = 2u;

template <typename T, int D, bool RING, int RS, int BN>
YOCO_DEV void fill_rows_without_node(const Params &p, int w, int warps, unsigned int *status) {
    if (RING && !p.n_nodes) return;   // every node is there
    const int lane = threadIdx.x & 31, pairs = p.B * p.N;
    for (int i = (int)blockIdx.x * warps + w; i < pairs; i += (int)gridDim.x * warps) {
        const int b = i / p.N, node = i - b * p.N;
        const Seq s = sequence<RING, RS, BN>(p, b);
        if (!s.ok && node == 0 && lane == 0) atomicOr(status, kStatusBadSequence);
        if (node < s.n) continue;
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.o) + (int64_t)i * p.Hq * D);
        for (int c = lane; c < p.Hq * (D * (int)sizeof(T) / 16); c += 32) dst[c] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int h = lane; h < p.Hq; h += 32) p.lse[((int64_t)b * p.Hq + h) * p.N + node] = -INFINITY;
    }
}

// ------------------------------------------------------------- visibility
// pos - window < at <= pos, whatever the two positions are.
YOCO_DEV bool in_window(int64_t pos, int64_t at, int32_t window) {
    return at <= pos && (uint64_t)pos - (uint64_t)at < (uint64_t)window;
}

// The nodes that node i of n sees, one bit each: the mask's (a chain's without
// one), of those that exist, and for a ring those inside i's window.
template <bool RING>
YOCO_DEV uint64_t visible_nodes(const Params &p, int b, int n, int i) {
    const int64_t at = (int64_t)b * p.N;
    uint64_t w = p.mask ? p.mask[at + i] : (2ull << i) - 1;
    if (n < 64) w &= (1ull << n) - 1;
    if (RING) {
        const int64_t pos = p.node_pos[at + i];
        for (int j = 0; j < n; ++j)
            if (!in_window(pos, p.node_pos[at + j], p.window)) w &= ~(1ull << j);
    }
    return w;
}

// The stored positions that a node at position pos sees in the ring: s >= 0 and
// pos - window < s < pos, kept as the 32-bit range (lo, hi].
struct RingBounds {
    int lo, hi;
    YOCO_DEV bool sees(int s) const { return (unsigned)s - (unsigned)lo - 1u < (unsigned)hi - (unsigned)lo; }
};
YOCO_DEV RingBounds ring_bounds(int64_t pos, int32_t window) {
    if (pos <= 0) return {-1, -1};
    const int64_t lo = sched::max64(pos - window, -1), hi = sched::min64(pos - 1, INT32_MAX);
    return {(int)sched::min64(lo, INT32_MAX), (int)hi};
}

inline Params make_params(const TreeArgs &a, const TreePlan &pl) {
    Params p;
    p.q = a.q; p.k_nodes = a.k_nodes; p.v_nodes = a.v_nodes; p.k = a.k; p.v = a.v;
    p.seq_start = a.seq_start; p.seq_len = a.seq_len; p.slot_pos = a.slot_pos; p.node_pos = a.node_pos;
    p.mask = a.mask; p.n_nodes = a.n_nodes;
    p.B = a.B; p.N = a.N; p.Hq = a.Hq; p.Hkv = a.Hkv; p.window = a.window;
    p.lg = a.Hq / a.Hkv == 8 ? 3 : a.Hq / a.Hkv == 4 ? 2 : a.Hq / a.Hkv == 2 ? 1 : 0;
    p.heads = pl.heads; p.groups = pl.groups; p.cluster = pl.cluster;
    p.cache_rows = a.cache_rows; p.max_len = a.max_len;
    p.scale_log2 = a.scale * kLog2e;
    p.o = a.o; p.lse = a.lse;
    unsigned char *ws = static_cast<unsigned char *>(a.ws);
    p.prefix = reinterpret_cast<int32_t *>(ws);
    p.ws_ml = reinterpret_cast<float2 *>(ws + pl.ml_off);
    p.ws_o = reinterpret_cast<float4 *>(ws + pl.o_off);
    return p;
}

}  // namespace tree
}  // namespace yoco
