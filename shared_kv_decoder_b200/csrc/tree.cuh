// What the tree-decode kernels share: their parameters, how the work is dealt
// to the CTAs, and which keys a drafted token sees.
//
// Work.  A "stream" is the rows of one (sequence, row block, KV head): RS rows
// of the row order r = node * G + head-in-group (G = Hq / Hkv), against that
// sequence's keys in tiles of BN -- first the context (the cache's rows, or the
// ring's slots), then one tile with the drafted nodes' own keys.  All streams'
// tiles are numbered sequence by sequence (row block outermost, then KV head,
// then tile), and CTA c of G takes the range [c T / G, (c + 1) T / G) of the T
// tiles (G no more than T, so that none is empty): every CTA gets the same
// number to within one whatever the lengths are, and a long stream is shared by as many CTAs as it has work for.  Row
// blocks of one sequence follow one another, so the CTAs that read the same
// keys for different rows do it at about the same time (from L2).  A CTA's
// part of a stream is a segment.  A stream that one CTA has whole is finished
// by it; of one that is shared, each CTA leaves a partial (m, l, unnormalised
// o) in the workspace, slot 0 for the segment its range opens with, slot 1 for
// the one it ends with, and tree_merge_kernel joins them.
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
    int32_t window;                      // 0: cache
    int64_t cache_rows, max_len;
    float scale_log2;
    void *o;                             // [B, N, Hq, D]
    float *lse;                          // [B, Hq, N] or null
    int64_t *prefix;                     // workspace: first tile of each sequence, then the total
    float2 *ws_ml;                       // workspace: [2 grid][RS]
    float *ws_o;                         // workspace: [2 grid][RS][D]
};

// One sequence: its nodes (0 when it has none or is out of range), context
// keys, context tiles and streams.
struct Seq {
    int n, n_ctx_tiles, n_rt;
    int64_t ctx, row0;
    bool ok;
    YOCO_DEV int64_t tiles(int Hkv) const { return (int64_t)n_rt * Hkv * (n_ctx_tiles + 1); }
};

template <bool RING, int RS, int BN>
YOCO_DEV Seq sequence(const Params &p, int b) {
    Seq s;
    const int G = p.Hq / p.Hkv;
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
    s.n_ctx_tiles = s.ok ? (int)((s.ctx + BN - 1) / BN) : 0;
    s.n_rt = (s.n * G + RS - 1) / RS;
    return s;
}

YOCO_DEV int64_t range_start(int64_t T, int64_t c, int64_t grid) { return c * T / grid; }
YOCO_DEV int64_t range_owner(int64_t T, int64_t x, int64_t grid) { return ((x + 1) * grid - 1) / T; }

// Where a CTA's range starts: the range [x, end), the sequence that holds x and
// that sequence's first tile.  Run by one whole warp; CTA 0 also leaves the
// prefix of tile counts in the workspace for the merge.
struct Range {
    int64_t x, end, base;
    int b;
};

template <bool RING, int RS, int BN>
YOCO_DEV Range find_range(const Params &p) {
    const int lane = threadIdx.x & 31;
    int64_t T = 0;
    for (int b = lane; b < p.B; b += 32) T += sequence<RING, RS, BN>(p, b).tiles(p.Hkv);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
    Range r;
    const int64_t grid = sched::min64(T, gridDim.x);
    r.x = r.end = T;
    if (blockIdx.x < grid) {
        r.x = range_start(T, blockIdx.x, grid);
        r.end = range_start(T, blockIdx.x + 1, grid);
    }
    r.b = p.B;
    r.base = T;
    bool found = r.x >= r.end;
    int64_t base = 0;
    for (int b0 = 0; b0 < p.B && (!found || blockIdx.x == 0); b0 += 32) {
        const int b = b0 + lane;
        const int64_t cnt = b < p.B ? sequence<RING, RS, BN>(p, b).tiles(p.Hkv) : 0;
        int64_t incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, base + incl > r.x);
        if (!found && hit) {
            const int src = __ffs(hit) - 1;
            r.b = b0 + src;
            r.base = __shfl_sync(0xffffffffu, base + incl - cnt, src);
            found = true;
        }
        if (blockIdx.x == 0 && b < p.B) p.prefix[b] = base + incl - cnt;
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (blockIdx.x == 0 && lane == 0) p.prefix[p.B] = T;
    return r;
}

// A segment: tiles [t0, t1) of one stream.
struct Seg {
    int b, rt, g;        // sequence, row block, KV head
    int n, n_ctx_tiles;  // its nodes and context tiles (tile n_ctx_tiles holds the nodes)
    int t0, t1;
    int64_t ctx, row0;
    bool whole;          // the CTA has the whole stream
    int slot;            // partial slot otherwise
};

// Steps through a CTA's segments.  Every role of a kernel runs its own copy.
template <bool RING, int RS, int BN>
struct SegIter {
    Range r;
    int64_t x0;
    Seq s;
    int64_t tiles;
    YOCO_DEV SegIter(const Params &p, const Range &range) : r(range), x0(range.x), tiles(0) {
        if (r.x < r.end) {
            s = sequence<RING, RS, BN>(p, r.b);
            tiles = s.tiles(p.Hkv);
        }
    }
    YOCO_DEV bool next(const Params &p, Seg &g) {
        if (r.x >= r.end) return false;
        while (r.x >= r.base + tiles) {
            r.base += tiles;
            s = sequence<RING, RS, BN>(p, ++r.b);
            tiles = s.tiles(p.Hkv);
        }
        const int nt = s.n_ctx_tiles + 1;
        const int64_t off = r.x - r.base;
        const int stream = (int)(off / nt);
        g.b = r.b;
        g.rt = stream / p.Hkv;
        g.g = stream - g.rt * p.Hkv;
        g.n = s.n;
        g.n_ctx_tiles = s.n_ctx_tiles;
        g.ctx = s.ctx;
        g.row0 = s.row0;
        g.t0 = (int)(off - (int64_t)stream * nt);
        g.t1 = (int)sched::min64(nt, g.t0 + (r.end - r.x));
        g.whole = g.t0 == 0 && g.t1 == nt;
        g.slot = r.x == x0 ? 0 : 1;
        r.x += g.t1 - g.t0;
        return true;
    }
};

// ------------------------------------------------------------- visibility
// The nodes that node i of n sees, one bit each: the mask's (a chain's without
// one), of those that exist, and for a ring those inside i's window.
template <bool RING>
YOCO_DEV uint64_t visible_nodes(const Params &p, int b, int n, int i) {
    const int64_t at = (int64_t)b * p.N;
    uint64_t w = p.mask ? p.mask[at + i] : (2ull << i) - 1;
    if (n < 64) w &= (1ull << n) - 1;
    if (RING) {
        const uint64_t pos = (uint64_t)p.node_pos[at + i];
        for (int j = 0; j < n; ++j)
            if (pos - (uint64_t)p.node_pos[at + j] >= (uint64_t)p.window) w &= ~(1ull << j);
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
    p.cache_rows = a.cache_rows; p.max_len = a.max_len;
    p.scale_log2 = a.scale * kLog2e;
    p.o = a.o; p.lse = a.lse;
    unsigned char *ws = static_cast<unsigned char *>(a.ws);
    p.prefix = reinterpret_cast<int64_t *>(ws);
    p.ws_ml = reinterpret_cast<float2 *>(ws + pl.ml_off);
    p.ws_o = reinterpret_cast<float *>(ws + pl.o_off);
    return p;
}

}  // namespace tree
}  // namespace yoco
