// The accepted path of a drafted tree, written into the shared cache or the
// self-decoder's ring (sm_100a).
//
// path[b][0 .. n_path[b]) names the nodes of sequence b that were accepted, in
// order.  Cache: node path[j]'s K / V become row seq_start + seq_len + j.
// Ring: they go to slot p mod window, p the node's position, and slot_pos
// there becomes p; of two that share a slot the later one of the path stays,
// as if they had been pushed one by one.  A sequence whose arguments are out
// of range is left as it is and reported.
//
// A copy of a few rows: bound by launch and memory latency.  One CTA copies the
// rows of one sequence's K or V (or a part of them), kept in flight four
// 16-byte chunks a thread at a time.
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "schedule.h"

namespace yoco {

// Bit 1: a sequence's arguments were out of range.
static __device__ unsigned int g_status_commit;
constexpr unsigned int kStatusBadSequence = 2u;

namespace {

constexpr int kCommitThreads = 256;
constexpr int kUnroll = 4;

}  // namespace

// grid (sequence, K / V, part)
template <bool RING>
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const CommitArgs a) {
    __shared__ int s_node[kTreeMaxNodes];
    __shared__ int64_t s_row[kTreeMaxNodes];   // -1: another node of the path has the slot
    __shared__ int s_slot[kTreeMaxNodes];
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x, tid = threadIdx.x;
    const bool first = blockIdx.y == 0 && blockIdx.z == 0;
    const int n = a.n_path[b];
    bool ok = n >= 0 && n <= a.N;
    int64_t start = 0, len = 0;
    if (!RING) {
        start = a.seq_start[b];
        len = a.seq_len[b];
        const int64_t cap = a.seq_cap ? a.seq_cap[b] : INT32_MAX;
        ok = ok && len >= 0 && start >= 0 && len + n <= cap && len + n <= INT32_MAX &&
             start <= a.cache_rows - (len + n);
    }
    int64_t pos = 0;
    if (ok && tid < n) {
        const int node = a.path[(int64_t)b * a.N + tid];
        ok = node >= 0 && node < a.N;
        if (RING && ok) {
            pos = a.node_pos[(int64_t)b * a.N + node];
            ok = pos >= 0 && pos <= INT32_MAX;
            s_slot[tid] = ok ? (int)(pos % a.window) : -1;
        }
        s_node[tid] = node;
        s_row[tid] = start + len + tid;
    }
    ok = __syncthreads_and(ok);
    if (RING) {
        if (ok && tid < n) {
            const int slot = s_slot[tid];
            bool last = true;
            for (int j = tid + 1; j < n; ++j) last &= s_slot[j] != slot;
            s_row[tid] = last ? (int64_t)b * a.window + slot : -1;
            if (last && first) a.slot_pos[(int64_t)b * a.window + slot] = (int)pos;
        }
        __syncthreads();
    }
    if (first && tid == 0) {
        if (!ok) atomicOr(&g_status_commit, kStatusBadSequence);
        if (!RING) a.new_len[b] = a.seq_len[b] + (ok ? n : 0);
    }
    if (!ok) return;
    const uint4 *src = static_cast<const uint4 *>(blockIdx.y == 0 ? a.k_nodes : a.v_nodes);
    uint4 *dst = static_cast<uint4 *>(blockIdx.y == 0 ? a.k : a.v);
    const int chunks = (int)(a.row_bytes / 16);
    const int total = n * chunks, stride = kCommitThreads * gridDim.z;
    for (int c0 = blockIdx.z * kCommitThreads + tid; c0 < total; c0 += kUnroll * stride) {
        uint4 x[kUnroll];
        int64_t to[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int c = c0 + u * stride;
            to[u] = -1;
            if (c >= total) continue;
            const int j = c / chunks, e = c - j * chunks;
            if (s_row[j] < 0) continue;
            to[u] = s_row[j] * chunks + e;
            x[u] = src[((int64_t)b * a.N + s_node[j]) * chunks + e];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (to[u] >= 0) dst[to[u]] = x[u];
    }
}

cudaError_t launch_commit(const CommitArgs &a, cudaStream_t st) {
    // parts: enough for every chunk of a full path to be in flight at once, no
    // more CTAs than a few waves
    const int64_t chunks = (int64_t)a.N * (a.row_bytes / 16);
    if (chunks > INT32_MAX / 2) return cudaErrorNotSupported;   // counted in 32 bits
    const int64_t parts = (chunks + kCommitThreads * kUnroll - 1) / (kCommitThreads * kUnroll);
    const int64_t room = std::max<int64_t>(1, (int64_t)4 * device_sm_count() / std::max(1, a.B));
    const dim3 grid((unsigned)a.B, 2, (unsigned)std::max<int64_t>(1, std::min(parts, room)));
    note_launches(1);
    return launch_pdl(a.window > 0 ? tree_commit_kernel<true> : tree_commit_kernel<false>, grid, dim3(kCommitThreads), 0,
                      st, a);
}

unsigned int read_and_clear_status_commit() {
    unsigned int h = 0, z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_commit, sizeof(h)) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_status_commit, &z, sizeof(z));
    return h;
}

}  // namespace yoco
