// C ABI of libyoco.so (declared in include/yoco.h): argument validation and
// dispatch to the sm_100a kernels.  Nothing is launched unless every check
// passes; the library never allocates device memory and never synchronises
// the host on a hot call.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "../../include/yoco.h"
#include "launch.h"
#include "schedule.h"

using namespace yoco;

namespace yoco {
static std::atomic<uint64_t> g_launches{0};
void note_launches(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }
}  // namespace yoco

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptr(const void *p) { return p != nullptr && aligned16(p); }
bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}
bool ok_opt(const void *p) { return p == nullptr || aligned16(p); }
// The decode kernels address cache rows with 32-bit TMA coordinates.
bool ok_cache_rows(int64_t rows) { return rows >= 1 && rows <= INT32_MAX; }

yoco_status check_cfg(const yoco_attn_cfg *cfg) {
    if (!cfg) return YOCO_ERR_INVALID;
    if (cfg->Hq < 1 || cfg->Hkv < 1 || cfg->Hq % cfg->Hkv != 0) return YOCO_ERR_INVALID;
    if (cfg->dtype != YOCO_BF16 && cfg->dtype != YOCO_FP32) return YOCO_ERR_INVALID;
    if (!(cfg->scale >= 0.f) || isinf(cfg->scale)) return YOCO_ERR_INVALID;
    if (cfg->D != 64 && cfg->D != 128) return YOCO_ERR_UNSUPPORTED;
    const int G = cfg->Hq / cfg->Hkv;
    if (G != 1 && G != 2 && G != 4 && G != 8) return YOCO_ERR_UNSUPPORTED;
    return YOCO_OK;
}

float eff_scale(const yoco_attn_cfg *cfg) {
    return cfg->scale > 0.f ? cfg->scale : 1.0f / sqrtf((float)cfg->D);
}

yoco_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return YOCO_OK;
    if (e == cudaErrorNotSupported) return YOCO_ERR_UNSUPPORTED;
    return YOCO_ERR_CUDA;
}

// Projection dispatch: the tensor-core kernel where it applies, else CUDA cores.
yoco_status run_linear(const LinearArgs &a, cudaStream_t s) {
    const cudaError_t e = launch_linear_tc(a, s);
    if (e != cudaErrorNotSupported) return from_cuda(e);
    cudaGetLastError();
    return from_cuda(launch_linear_simt(a, s));
}

// Attention prefill dispatch: bf16 goes to a tcgen05 kernel -- two query
// heads per CTA when the group size is even, else one; fp32 (and any bf16
// shape those kernels were not built for) to the CUDA-core kernel.
yoco_status run_prefill(const PrefillArgs &a, cudaStream_t s) {
    if (a.dtype == kBF16) {
        cudaError_t e = launch_prefill_pair(a, s);
        if (e != cudaErrorNotSupported) return from_cuda(e);
        cudaGetLastError();
        e = launch_prefill_tc(a, s);
        if (e != cudaErrorNotSupported) return from_cuda(e);
        cudaGetLastError();
    }
    return from_cuda(launch_prefill_simt(a, s));
}

}  // namespace

extern "C" {

const char *yoco_version(void) { return "yoco-b200 0.1 (sm_100a)"; }

uint64_t yoco_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

const char *yoco_status_string(yoco_status s) {
    switch (s) {
        case YOCO_OK: return "ok";
        case YOCO_ERR_INVALID: return "invalid argument";
        case YOCO_ERR_UNSUPPORTED: return "unsupported shape or type";
        case YOCO_ERR_CUDA: return "CUDA error";
        case YOCO_ERR_WORKSPACE: return "workspace missing or too small";
        case YOCO_ERR_TIMEOUT: return "device wait timed out";
    }
    return "unknown status";
}

yoco_status yoco_kv_project_blend(const void *x, int64_t n_tok, int32_t d_model, const void *w_kv,
                                  int32_t apply_ln, float ln_eps, const void *k_base,
                                  const void *v_base, float w_k, float w_v,
                                  const int64_t *dst_rows, void *k_out, void *v_out,
                                  const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (n_tok < 0 || d_model < 1 || !(ln_eps > 0.f) || !isfinite(w_k) || !isfinite(w_v))
        return YOCO_ERR_INVALID;
    if (n_tok == 0) return YOCO_OK;
    if (!ok_ptr(x) || !ok_ptr(w_kv) || !ok_ptr(k_out) || !ok_ptr(v_out) || !ok_opt(k_base) ||
        !ok_opt(v_base) || !ok_opt(dst_rows))
        return YOCO_ERR_INVALID;
    if ((int64_t)d_model * dtype_bytes(cfg->dtype) % 16 != 0) return YOCO_ERR_INVALID;
    LinearArgs a;
    a.x = x; a.w = w_kv; a.n = n_tok; a.d_in = d_model;
    a.d_out = 2 * cfg->Hkv * cfg->D; a.split_col = cfg->Hkv * cfg->D;
    a.apply_ln = apply_ln ? 1 : 0; a.eps = ln_eps;
    a.out0 = k_out; a.out1 = v_out; a.base0 = k_base; a.base1 = v_base;
    a.w0 = w_k; a.w1 = w_v; a.dst_rows = dst_rows; a.dtype = cfg->dtype;
    return run_linear(a, stream);
}

yoco_status yoco_linear(const void *x, int64_t n, int32_t d_in, const void *w, int32_t d_out,
                        int32_t apply_ln, float ln_eps, const void *base, float base_w, void *out,
                        int32_t dtype, cudaStream_t stream) {
    if (dtype != YOCO_BF16 && dtype != YOCO_FP32) return YOCO_ERR_INVALID;
    if (n < 0 || d_in < 1 || d_out < 1 || !(ln_eps > 0.f) || !isfinite(base_w))
        return YOCO_ERR_INVALID;
    if (n == 0) return YOCO_OK;
    if (!ok_ptr(x) || !ok_ptr(w) || !ok_ptr(out) || !ok_opt(base)) return YOCO_ERR_INVALID;
    LinearArgs a;
    a.x = x; a.w = w; a.n = n; a.d_in = d_in; a.d_out = d_out; a.split_col = d_out;
    a.apply_ln = apply_ln ? 1 : 0; a.eps = ln_eps;
    a.out0 = out; a.out1 = nullptr; a.base0 = base; a.base1 = nullptr;
    a.w0 = base_w; a.w1 = 0.f; a.dst_rows = nullptr; a.dtype = dtype;
    return run_linear(a, stream);
}

yoco_status yoco_swa_prefill(const void *q, const void *k, const void *v, int32_t B, int64_t T,
                             int32_t window, void *o, float *lse, void *ring_k, void *ring_v,
                             int32_t *slot_pos, const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || T < 0 || window < 1) return YOCO_ERR_INVALID;
    const int rings = (ring_k != nullptr) + (ring_v != nullptr) + (slot_pos != nullptr);
    if (rings != 0 && rings != 3) return YOCO_ERR_INVALID;
    if (B == 0) return YOCO_OK;
    if (T > 0 && (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o) || !ok_opt(lse)))
        return YOCO_ERR_INVALID;
    if (rings == 3 && (!ok_ptr(ring_k) || !ok_ptr(ring_v) || !ok_ptr(slot_pos)))
        return YOCO_ERR_INVALID;
    if (T > 0) {
        PrefillArgs a;
        a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
        a.B = B; a.Tq = T; a.Tkv = T; a.q_pos0 = 0; a.window = window;
        a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.D = cfg->D; a.dtype = cfg->dtype;
        a.scale = eff_scale(cfg);
        st = run_prefill(a, stream);
        if (st != YOCO_OK) return st;
    }
    if (rings == 3)
        return from_cuda(launch_ring_fill(k, v, B, T, window, cfg->Hkv, cfg->D, cfg->dtype, ring_k,
                                          ring_v, slot_pos, stream));
    return YOCO_OK;
}

yoco_status yoco_cross_prefill(const void *q, const void *k, const void *v, int32_t B, int64_t Tq,
                               int64_t Tkv, int64_t q_pos0, void *o, float *lse,
                               const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || Tq < 0 || Tkv < 0 || q_pos0 < 0 || q_pos0 + Tq > Tkv) return YOCO_ERR_INVALID;
    if (B == 0 || Tq == 0) return YOCO_OK;
    if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o) || !ok_opt(lse)) return YOCO_ERR_INVALID;
    PrefillArgs a;
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    a.B = B; a.Tq = Tq; a.Tkv = Tkv; a.q_pos0 = q_pos0; a.window = 0;
    a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.D = cfg->D; a.dtype = cfg->dtype;
    a.scale = eff_scale(cfg);
    return run_prefill(a, stream);
}

yoco_status yoco_attention_prefill(const void *q, const void *k, const void *v, int32_t B, int64_t Tq,
                                   int64_t Tkv, int64_t q_pos0, int32_t window, void *o, float *lse,
                                   const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || Tq < 0 || Tkv < 0 || q_pos0 < 0 || q_pos0 + Tq > Tkv || window < 0) return YOCO_ERR_INVALID;
    if (B == 0 || Tq == 0) return YOCO_OK;
    if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o) || !ok_opt(lse)) return YOCO_ERR_INVALID;
    PrefillArgs a;
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    a.B = B; a.Tq = Tq; a.Tkv = Tkv; a.q_pos0 = q_pos0; a.window = window;
    a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.D = cfg->D; a.dtype = cfg->dtype;
    a.scale = eff_scale(cfg);
    return run_prefill(a, stream);
}

size_t yoco_cross_decode_workspace_size(int32_t B, int64_t max_len, const yoco_attn_cfg *cfg) {
    if (check_cfg(cfg) != YOCO_OK) return 0;
    DecodePlan pl;
    if (!make_decode_plan(B, max_len, cfg->Hq, cfg->Hkv, cfg->D, cfg->dtype, &pl)) return 0;
    return pl.ws_bytes;
}

size_t yoco_swa_decode_workspace_size(int32_t B, int32_t window, const yoco_attn_cfg *cfg) {
    return yoco_cross_decode_workspace_size(B, window, cfg);
}

yoco_status yoco_cross_decode(const void *q, const void *k_cache, const void *v_cache,
                              int64_t cache_rows, const int64_t *seq_start, const int32_t *seq_len,
                              int32_t B, int64_t max_len, void *o, float *lse, void *workspace,
                              size_t ws_bytes, const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || max_len < 1 || !ok_cache_rows(cache_rows)) return YOCO_ERR_INVALID;
    if (B == 0) return YOCO_OK;
    if (!ok_ptr(q) || !ok_ptr(k_cache) || !ok_ptr(v_cache) || !ok_ptr(seq_start) ||
        !seq_len || !ok_ptr(o) || !ok_opt(lse))
        return YOCO_ERR_INVALID;
    DecodePlan pl;
    if (!make_decode_plan(B, max_len, cfg->Hq, cfg->Hkv, cfg->D, cfg->dtype, &pl))
        return YOCO_ERR_UNSUPPORTED;
    if (!workspace || !aligned16(workspace) || ws_bytes < pl.ws_bytes) return YOCO_ERR_WORKSPACE;
    DecodeArgs a;
    a.q = q; a.k = k_cache; a.v = v_cache; a.seq_start = seq_start; a.seq_len = seq_len;
    a.slot_pos = nullptr; a.pos = nullptr; a.window = 0; a.k_new = a.v_new = nullptr;
    a.cache_rows = cache_rows; a.max_len = max_len;
    a.B = B; a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.D = cfg->D; a.dtype = cfg->dtype;
    a.scale = eff_scale(cfg); a.o = o; a.lse = lse; a.ws = workspace;
    return from_cuda(launch_decode(a, pl, stream));
}

yoco_status yoco_swa_decode(const void *q, const void *k_new, const void *v_new,
                            const int64_t *pos, int32_t B, int32_t window, void *ring_k,
                            void *ring_v, int32_t *slot_pos, void *o, void *workspace,
                            size_t ws_bytes, const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || window < 1) return YOCO_ERR_INVALID;
    if (B == 0) return YOCO_OK;
    if (!ok_ptr(q) || !ok_ptr(k_new) || !ok_ptr(v_new) || !ok_ptr(pos) || !ok_ptr(ring_k) ||
        !ok_ptr(ring_v) || !ok_ptr(slot_pos) || !ok_ptr(o))
        return YOCO_ERR_INVALID;
    DecodePlan pl;
    if (!make_decode_plan(B, window, cfg->Hq, cfg->Hkv, cfg->D, cfg->dtype, &pl))
        return YOCO_ERR_UNSUPPORTED;
    if (!workspace || !aligned16(workspace) || ws_bytes < pl.ws_bytes) return YOCO_ERR_WORKSPACE;
    // the window read skips the new token's slot; the merge adds the new
    // token and writes it into the ring (no separate ring-write kernel)
    DecodeArgs a;
    a.q = q; a.k = ring_k; a.v = ring_v; a.seq_start = nullptr; a.seq_len = nullptr;
    a.slot_pos = slot_pos; a.pos = pos; a.window = window;
    a.k_new = k_new; a.v_new = v_new;
    a.cache_rows = (int64_t)B * window; a.max_len = window;
    a.B = B; a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.D = cfg->D; a.dtype = cfg->dtype;
    a.scale = eff_scale(cfg); a.o = o; a.lse = nullptr; a.ws = workspace;
    // bf16: one clustered launch (window read, merge, new token, ring write);
    // other shapes: the split kernel and the merge
    const cudaError_t e = launch_ring_decode(a, stream);
    if (e != cudaErrorNotSupported) return from_cuda(e);
    return from_cuda(launch_decode(a, pl, stream));
}

size_t yoco_swa_decode_step_workspace_size(int32_t B, int32_t window, const yoco_attn_cfg *cfg) {
    if (check_cfg(cfg) != YOCO_OK || B < 0 || window < 1) return 0;
    const size_t dws = yoco_swa_decode_workspace_size(B, window, cfg);
    if (dws == 0) return 0;
    const size_t kv = ((size_t)B * cfg->Hkv * cfg->D * dtype_bytes(cfg->dtype) + 15) / 16 * 16;
    return 2 * kv + dws;
}

yoco_status yoco_swa_decode_step(const void *x, int32_t d_model, const void *w_kv, int32_t apply_ln,
                                 float ln_eps, const void *k_base, const void *v_base, float w_k, float w_v,
                                 const void *q, const int64_t *pos, int32_t B, int32_t window, void *ring_k,
                                 void *ring_v, int32_t *slot_pos, void *o, void *k_out, void *v_out,
                                 void *workspace, size_t ws_bytes, const yoco_attn_cfg *cfg,
                                 cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || window < 1 || d_model < 1 || !(ln_eps > 0.f) || !isfinite(w_k) || !isfinite(w_v))
        return YOCO_ERR_INVALID;
    if (B == 0) return YOCO_OK;
    if (!ok_ptr(x) || !ok_ptr(w_kv) || !ok_ptr(q) || !ok_ptr(pos) || !ok_ptr(ring_k) || !ok_ptr(ring_v) ||
        !ok_ptr(slot_pos) || !ok_ptr(o) || !ok_opt(k_base) || !ok_opt(v_base) || !ok_opt(k_out) ||
        !ok_opt(v_out))
        return YOCO_ERR_INVALID;
    if ((int64_t)d_model * dtype_bytes(cfg->dtype) % 16 != 0) return YOCO_ERR_INVALID;
    DecodePlan pl;
    if (!make_decode_plan(B, window, cfg->Hq, cfg->Hkv, cfg->D, cfg->dtype, &pl)) return YOCO_ERR_UNSUPPORTED;
    const size_t need = yoco_swa_decode_step_workspace_size(B, window, cfg);
    if (!workspace || !aligned16(workspace) || need == 0 || ws_bytes < need) return YOCO_ERR_WORKSPACE;
    // the projection into k_out / v_out (or the workspace), then the window
    // decode.  bf16 few-token projections stream their weights through
    // registers; after that kernel the window decode runs in its compact
    // layout (four CTAs a head), the faster one there.
    const size_t kvb = ((size_t)B * cfg->Hkv * cfg->D * dtype_bytes(cfg->dtype) + 15) / 16 * 16;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    void *kn = k_out ? k_out : ws;
    void *vn = v_out ? v_out : ws + kvb;
    LinearArgs la;
    la.x = x; la.w = w_kv; la.n = B; la.d_in = d_model;
    la.d_out = 2 * cfg->Hkv * cfg->D; la.split_col = cfg->Hkv * cfg->D;
    la.apply_ln = apply_ln ? 1 : 0; la.eps = ln_eps;
    la.out0 = kn; la.out1 = vn; la.base0 = k_base; la.base1 = v_base;
    la.w0 = w_k; la.w1 = w_v; la.dst_rows = nullptr; la.dtype = cfg->dtype;
    cudaError_t e = launch_linear_few_reg(la, stream);
    const bool compact = e == cudaSuccess;
    if (e == cudaErrorNotSupported) {
        cudaGetLastError();
        st = run_linear(la, stream);
        if (st != YOCO_OK) return st;
    } else if (e != cudaSuccess) {
        return from_cuda(e);
    }
    DecodeArgs a;
    a.q = q; a.k = ring_k; a.v = ring_v; a.seq_start = nullptr; a.seq_len = nullptr;
    a.slot_pos = slot_pos; a.pos = pos; a.window = window;
    a.k_new = kn; a.v_new = vn;
    a.cache_rows = (int64_t)B * window; a.max_len = window;
    a.B = B; a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.D = cfg->D; a.dtype = cfg->dtype;
    a.scale = eff_scale(cfg); a.o = o; a.lse = nullptr; a.ws = ws + 2 * kvb;
    const cudaError_t e2 = launch_ring_decode(a, stream, compact);
    if (e2 != cudaErrorNotSupported) return from_cuda(e2);
    cudaGetLastError();
    return from_cuda(launch_decode(a, pl, stream));
}

int64_t yoco_kv_i8_row_bytes(const yoco_attn_cfg *cfg) {
    if (!cfg || cfg->Hkv < 1 || (cfg->D != 64 && cfg->D != 128)) return 0;
    return i8_row_bytes(cfg->Hkv, cfg->D);
}

yoco_status yoco_kv_quantize_i8(const void *k, const void *v, int64_t n_tok, const int64_t *dst_rows, void *k_i8,
                                void *v_i8, const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (n_tok < 0) return YOCO_ERR_INVALID;
    if (n_tok == 0) return YOCO_OK;
    if (!ok_ptr(k) || !ok_ptr(v) || !ok_opt(dst_rows) || !ok_ptr(k_i8) || !ok_ptr(v_i8)) return YOCO_ERR_INVALID;
    return from_cuda(launch_kv_quantize_i8(k, v, n_tok, cfg->Hkv, cfg->D, cfg->dtype, dst_rows, k_i8, v_i8, stream));
}

yoco_status yoco_cross_decode_i8(const void *q, const void *k_i8, const void *v_i8, int64_t cache_rows,
                                 const int64_t *seq_start, const int32_t *seq_len, int32_t B, int64_t max_len,
                                 void *o, float *lse, void *workspace, size_t ws_bytes, const yoco_attn_cfg *cfg,
                                 cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || max_len < 1 || !ok_cache_rows(cache_rows)) return YOCO_ERR_INVALID;
    if (B == 0) return YOCO_OK;
    if (!ok_ptr(q) || !ok_ptr(k_i8) || !ok_ptr(v_i8) || !ok_ptr(seq_start) || !seq_len || !ok_ptr(o) || !ok_opt(lse))
        return YOCO_ERR_INVALID;
    if (cfg->D != 128 || cfg->dtype != YOCO_BF16) return YOCO_ERR_UNSUPPORTED;
    DecodePlan pl;
    if (!make_decode_plan(B, max_len, cfg->Hq, cfg->Hkv, cfg->D, cfg->dtype, &pl)) return YOCO_ERR_UNSUPPORTED;
    if (!workspace || !aligned16(workspace) || ws_bytes < pl.ws_bytes) return YOCO_ERR_WORKSPACE;
    DecodeArgs a;
    a.q = q; a.k = k_i8; a.v = v_i8; a.seq_start = seq_start; a.seq_len = seq_len;
    a.slot_pos = nullptr; a.pos = nullptr; a.window = 0; a.k_new = a.v_new = nullptr;
    a.cache_rows = cache_rows; a.max_len = max_len;
    a.B = B; a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.D = cfg->D; a.dtype = cfg->dtype;
    a.scale = eff_scale(cfg); a.o = o; a.lse = lse; a.ws = workspace;
    return from_cuda(launch_decode_i8(a, pl, stream));
}

size_t yoco_gret_prefill_workspace_size(int32_t B, int64_t T, const yoco_attn_cfg *cfg) {
    if (check_cfg(cfg) != YOCO_OK || cfg->Hq != cfg->Hkv || cfg->dtype != YOCO_BF16) return 0;
    return gret_workspace_bytes(B, cfg->Hq, T, cfg->D);
}

yoco_status yoco_gret_prefill(const void *q, const void *k, const void *v, const float *g, int32_t B,
                              int64_t T, float tau, float *state, void *o, void *workspace, size_t ws_bytes,
                              const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (cfg->Hq != cfg->Hkv || B < 0 || T < 0 || !(tau > 0.f) || isinf(tau)) return YOCO_ERR_INVALID;
    if (B == 0 || T == 0) return YOCO_OK;
    if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(g) || !ok_opt(state) || !ok_ptr(o) ||
        !ok_opt(workspace))
        return YOCO_ERR_INVALID;
    if (cfg->dtype != YOCO_BF16) return YOCO_ERR_UNSUPPORTED;
    // a workspace enables the split over superchunks; one smaller than the
    // size query's answer is an error, a NULL one (or a size of 0) means no split
    const size_t need = gret_workspace_bytes(B, cfg->Hq, T, cfg->D);
    if (workspace && ws_bytes < need) return YOCO_ERR_WORKSPACE;
    GretArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.state = state; a.o = o;
    a.B = B; a.H = cfg->Hq; a.D = cfg->D; a.dtype = cfg->dtype; a.T = T;
    a.tau = tau; a.scale = eff_scale(cfg);
    a.ws = (workspace && need > 0) ? workspace : nullptr;
    return from_cuda(launch_gret_prefill(a, stream));
}

yoco_status yoco_gret_decode(const void *q, const void *k, const void *v, const float *g, int32_t B,
                             float tau, float *state, void *o, const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (cfg->Hq != cfg->Hkv || B < 0 || !(tau > 0.f) || isinf(tau)) return YOCO_ERR_INVALID;
    if (B == 0) return YOCO_OK;
    if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(g) || !ok_ptr(state) || !ok_ptr(o))
        return YOCO_ERR_INVALID;
    GretArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.state = state; a.o = o;
    a.B = B; a.H = cfg->Hq; a.D = cfg->D; a.dtype = cfg->dtype; a.T = 1;
    a.tau = tau; a.scale = eff_scale(cfg); a.ws = nullptr;
    return from_cuda(launch_gret_decode(a, stream));
}

yoco_status yoco_rope_init(yoco_rope_cfg *rope, int32_t rot_dim, int32_t layout, double theta, int32_t scaling,
                           double factor, double orig_len, double beta_fast, double beta_slow, double mscale) {
    if (!rope || rot_dim < 16 || rot_dim > 128 || rot_dim % 16 != 0) return YOCO_ERR_INVALID;
    if (layout != YOCO_ROPE_HALF && layout != YOCO_ROPE_INTERLEAVED) return YOCO_ERR_INVALID;
    if (scaling < YOCO_ROPE_NONE || scaling > YOCO_ROPE_BY_PARTS) return YOCO_ERR_INVALID;
    if (!(theta > 0.0) || isinf(theta) || !(mscale >= 0.0) || isinf(mscale)) return YOCO_ERR_INVALID;
    if (scaling != YOCO_ROPE_NONE && (!(factor >= 1.0) || isinf(factor))) return YOCO_ERR_INVALID;
    if (scaling == YOCO_ROPE_BY_PARTS &&
        (!(orig_len > 0.0) || isinf(orig_len) || !(beta_slow < beta_fast) || isinf(beta_slow) || isinf(beta_fast)))
        return YOCO_ERR_INVALID;
    constexpr double kTwoPi = 6.283185307179586476925;
    const double base = scaling == YOCO_ROPE_NTK ? theta * pow(factor, rot_dim / (rot_dim - 2.0)) : theta;
    rope->rot_dim = rot_dim;
    rope->layout = layout;
    rope->mscale = mscale > 0.0 ? mscale : scaling == YOCO_ROPE_BY_PARTS ? 0.1 * log(factor) + 1.0 : 1.0;
    for (int i = 0; i < 64; ++i) {
        double w = i < rot_dim / 2 ? pow(base, -2.0 * i / rot_dim) : 0.0;
        if (scaling == YOCO_ROPE_LINEAR) w /= factor;
        if (scaling == YOCO_ROPE_BY_PARTS) {
            const double r = orig_len * w / kTwoPi;
            const double g = std::min(1.0, std::max(0.0, (r - beta_slow) / (beta_fast - beta_slow)));
            w = g * w + (1.0 - g) * w / factor;
        }
        rope->inv_freq[i] = w;
    }
    return YOCO_OK;
}

yoco_status yoco_rope(const void *q, const void *k, int32_t B, int64_t T, const int64_t *pos, int64_t pos0,
                      int32_t backward, void *q_out, void *k_out, const yoco_rope_cfg *rope,
                      const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (!rope || rope->rot_dim < 16 || rope->rot_dim > 128 || rope->rot_dim % 16 != 0 ||
        (rope->layout != YOCO_ROPE_HALF && rope->layout != YOCO_ROPE_INTERLEAVED) || !isfinite(rope->mscale))
        return YOCO_ERR_INVALID;
    for (int i = 0; i < rope->rot_dim / 2; ++i)
        if (!isfinite(rope->inv_freq[i])) return YOCO_ERR_INVALID;
    if (rope->rot_dim > cfg->D) return YOCO_ERR_UNSUPPORTED;
    if (B < 0 || T < 0 || (T > 0 && B > INT64_MAX / T)) return YOCO_ERR_INVALID;
    if ((q != nullptr) != (q_out != nullptr) || (k != nullptr) != (k_out != nullptr)) return YOCO_ERR_INVALID;
    if (B == 0 || T == 0) return YOCO_OK;
    if ((!q && !k) || !ok_opt(q) || !ok_opt(k) || !ok_opt(q_out) || !ok_opt(k_out) || !ok_opt(pos))
        return YOCO_ERR_INVALID;
    if ((int64_t)cfg->Hq + cfg->Hkv > 1 << 24) return YOCO_ERR_UNSUPPORTED;   // a CTA counts its units in 32 bits
    const int64_t n = B * T, head = (int64_t)cfg->D * dtype_bytes(cfg->dtype);
    if (n > INT64_MAX / 2 / (cfg->Hq * head)) return YOCO_ERR_UNSUPPORTED;
    // in place, or apart from everything that is read
    const int64_t q_bytes = n * cfg->Hq * head, k_bytes = n * cfg->Hkv * head;
    if ((q_out != q && overlap(q_out, q_bytes, q, q_bytes)) || (k_out != k && overlap(k_out, k_bytes, k, k_bytes)) ||
        overlap(q_out, q_bytes, k, k_bytes) || overlap(k_out, k_bytes, q, q_bytes) ||
        overlap(q_out, q_bytes, k_out, k_bytes) || overlap(q_out, q_bytes, pos, 8 * n) ||
        overlap(k_out, k_bytes, pos, 8 * n))
        return YOCO_ERR_INVALID;
    RopeArgs a;
    a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out; a.pos = pos;
    a.n = n; a.T = T; a.pos0 = pos0;
    a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.D = cfg->D; a.dtype = cfg->dtype;
    a.rot_dim = rope->rot_dim; a.interleaved = rope->layout == YOCO_ROPE_INTERLEAVED; a.backward = backward != 0;
    a.mscale = (float)rope->mscale; a.inv_freq = rope->inv_freq;
    return from_cuda(launch_rope(a, stream));
}

size_t yoco_cross_decode_tree_workspace_size(int32_t B, int32_t N, int64_t max_len, const yoco_attn_cfg *cfg) {
    if (check_cfg(cfg) != YOCO_OK || B < 1 || N < 1 || N > kTreeMaxNodes || max_len < 0 || max_len > INT32_MAX) return 0;
    TreePlan pl;
    if (!make_tree_plan(B, N, max_len, cfg->Hq, cfg->Hkv, cfg->D, cfg->dtype, &pl)) return 0;
    return pl.ws_bytes;
}

size_t yoco_swa_decode_tree_workspace_size(int32_t B, int32_t N, int32_t window, const yoco_attn_cfg *cfg) {
    if (window < 1) return 0;
    return yoco_cross_decode_tree_workspace_size(B, N, window, cfg);
}

yoco_status yoco_cross_decode_tree(const void *q, const void *k_nodes, const void *v_nodes, const void *k_cache,
                                   const void *v_cache, int64_t cache_rows, const int64_t *seq_start,
                                   const int32_t *seq_len, const uint64_t *tree_mask, const int32_t *n_nodes,
                                   int32_t B, int32_t N, int64_t max_len, void *o, float *lse, void *workspace,
                                   size_t ws_bytes, const yoco_attn_cfg *cfg, cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || N < 1 || max_len < 0 || max_len > INT32_MAX || !ok_cache_rows(cache_rows)) return YOCO_ERR_INVALID;
    if (N > kTreeMaxNodes) return YOCO_ERR_UNSUPPORTED;
    if (B == 0) return YOCO_OK;
    if (!ok_ptr(q) || !ok_ptr(k_nodes) || !ok_ptr(v_nodes) || !ok_ptr(k_cache) || !ok_ptr(v_cache) ||
        !ok_ptr(seq_start) || !ok_ptr(seq_len) || !ok_opt(tree_mask) || !ok_opt(n_nodes) || !ok_ptr(o) || !ok_opt(lse))
        return YOCO_ERR_INVALID;
    TreePlan pl;
    if (!make_tree_plan(B, N, max_len, cfg->Hq, cfg->Hkv, cfg->D, cfg->dtype, &pl)) return YOCO_ERR_UNSUPPORTED;
    if (pl.ws_bytes > 0 && (!ok_ptr(workspace) || ws_bytes < pl.ws_bytes)) return YOCO_ERR_WORKSPACE;
    TreeArgs a;
    a.q = q; a.k_nodes = k_nodes; a.v_nodes = v_nodes; a.k = k_cache; a.v = v_cache;
    a.seq_start = seq_start; a.seq_len = seq_len; a.slot_pos = nullptr; a.node_pos = nullptr;
    a.mask = tree_mask; a.n_nodes = n_nodes; a.B = B; a.N = N;
    a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.D = cfg->D; a.dtype = cfg->dtype;
    a.window = 0; a.cache_rows = cache_rows; a.max_len = max_len;
    a.scale = eff_scale(cfg); a.o = o; a.lse = lse; a.ws = workspace;
    return from_cuda(launch_tree(a, pl, stream));
}

yoco_status yoco_swa_decode_tree(const void *q, const void *k_nodes, const void *v_nodes, const int64_t *node_pos,
                                 const uint64_t *tree_mask, const int32_t *n_nodes, int32_t B, int32_t N,
                                 int32_t window, const void *ring_k, const void *ring_v, const int32_t *slot_pos,
                                 void *o, float *lse, void *workspace, size_t ws_bytes, const yoco_attn_cfg *cfg,
                                 cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || N < 1 || window < 1) return YOCO_ERR_INVALID;
    if (N > kTreeMaxNodes) return YOCO_ERR_UNSUPPORTED;
    if (B == 0) return YOCO_OK;
    if (!ok_ptr(q) || !ok_ptr(k_nodes) || !ok_ptr(v_nodes) || !ok_ptr(node_pos) || !ok_opt(tree_mask) ||
        !ok_opt(n_nodes) || !ok_ptr(ring_k) || !ok_ptr(ring_v) || !ok_ptr(slot_pos) || !ok_ptr(o) || !ok_opt(lse))
        return YOCO_ERR_INVALID;
    TreePlan pl;
    if (!make_tree_plan(B, N, window, cfg->Hq, cfg->Hkv, cfg->D, cfg->dtype, &pl)) return YOCO_ERR_UNSUPPORTED;
    if (pl.ws_bytes > 0 && (!ok_ptr(workspace) || ws_bytes < pl.ws_bytes)) return YOCO_ERR_WORKSPACE;
    TreeArgs a;
    a.q = q; a.k_nodes = k_nodes; a.v_nodes = v_nodes; a.k = ring_k; a.v = ring_v;
    a.seq_start = nullptr; a.seq_len = nullptr; a.slot_pos = slot_pos; a.node_pos = node_pos;
    a.mask = tree_mask; a.n_nodes = n_nodes; a.B = B; a.N = N;
    a.Hq = cfg->Hq; a.Hkv = cfg->Hkv; a.D = cfg->D; a.dtype = cfg->dtype;
    a.window = window; a.cache_rows = (int64_t)B * window; a.max_len = window;
    a.scale = eff_scale(cfg); a.o = o; a.lse = lse; a.ws = workspace;
    return from_cuda(launch_tree(a, pl, stream));
}

yoco_status yoco_cross_tree_commit(const void *k_nodes, const void *v_nodes, const int32_t *path,
                                   const int32_t *n_path, int32_t B, int32_t N, void *k_cache, void *v_cache,
                                   int64_t cache_rows, const int64_t *seq_start, const int32_t *seq_len,
                                   const int32_t *seq_cap, int32_t *new_len, const yoco_attn_cfg *cfg,
                                   cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || N < 1 || !ok_cache_rows(cache_rows)) return YOCO_ERR_INVALID;
    if (N > kTreeMaxNodes) return YOCO_ERR_UNSUPPORTED;
    if (B == 0) return YOCO_OK;
    if (!ok_ptr(k_nodes) || !ok_ptr(v_nodes) || !ok_ptr(path) || !ok_ptr(n_path) || !ok_ptr(k_cache) ||
        !ok_ptr(v_cache) || !ok_ptr(seq_start) || !ok_ptr(seq_len) || !ok_opt(seq_cap) || !ok_ptr(new_len))
        return YOCO_ERR_INVALID;
    // other CTAs of a sequence read these while the first one writes new_len
    const int64_t per_seq = 4 * (int64_t)B;
    if (overlap(new_len, per_seq, seq_len, per_seq) || overlap(new_len, per_seq, n_path, per_seq) ||
        overlap(new_len, per_seq, seq_cap, per_seq) || overlap(new_len, per_seq, seq_start, 2 * per_seq) ||
        overlap(new_len, per_seq, path, per_seq * N))
        return YOCO_ERR_INVALID;
    CommitArgs a;
    a.k_nodes = k_nodes; a.v_nodes = v_nodes; a.path = path; a.n_path = n_path; a.B = B; a.N = N;
    a.row_bytes = (int64_t)cfg->Hkv * cfg->D * dtype_bytes(cfg->dtype);
    a.k = k_cache; a.v = v_cache; a.seq_start = seq_start; a.seq_len = seq_len; a.seq_cap = seq_cap;
    a.new_len = new_len; a.cache_rows = cache_rows;
    a.node_pos = nullptr; a.slot_pos = nullptr; a.window = 0;
    return from_cuda(launch_commit(a, stream));
}

yoco_status yoco_swa_tree_commit(const void *k_nodes, const void *v_nodes, const int64_t *node_pos,
                                 const int32_t *path, const int32_t *n_path, int32_t B, int32_t N, int32_t window,
                                 void *ring_k, void *ring_v, int32_t *slot_pos, const yoco_attn_cfg *cfg,
                                 cudaStream_t stream) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (B < 0 || N < 1 || window < 1) return YOCO_ERR_INVALID;
    if (N > kTreeMaxNodes) return YOCO_ERR_UNSUPPORTED;
    if (B == 0) return YOCO_OK;
    if (!ok_ptr(k_nodes) || !ok_ptr(v_nodes) || !ok_ptr(node_pos) || !ok_ptr(path) || !ok_ptr(n_path) ||
        !ok_ptr(ring_k) || !ok_ptr(ring_v) || !ok_ptr(slot_pos))
        return YOCO_ERR_INVALID;
    const int64_t per_seq = 4 * (int64_t)B, slots = per_seq * window;   // as above
    if (overlap(slot_pos, slots, n_path, per_seq) || overlap(slot_pos, slots, path, per_seq * N) ||
        overlap(slot_pos, slots, node_pos, 2 * per_seq * N))
        return YOCO_ERR_INVALID;
    CommitArgs a;
    a.k_nodes = k_nodes; a.v_nodes = v_nodes; a.path = path; a.n_path = n_path; a.B = B; a.N = N;
    a.row_bytes = (int64_t)cfg->Hkv * cfg->D * dtype_bytes(cfg->dtype);
    a.k = ring_k; a.v = ring_v; a.seq_start = nullptr; a.seq_len = nullptr; a.seq_cap = nullptr;
    a.new_len = nullptr; a.cache_rows = (int64_t)B * window;
    a.node_pos = node_pos; a.slot_pos = slot_pos; a.window = window;
    return from_cuda(launch_commit(a, stream));
}

yoco_status yoco_debug_tile_schedule(int32_t kind, const yoco_attn_cfg *cfg, int32_t B, int64_t Tq,
                                     int64_t Tkv, int64_t q_pos0, int32_t window,
                                     const int64_t *seq_start, const int32_t *seq_len, int64_t max_len,
                                     int32_t n_cta, int64_t *records, int64_t cap,
                                     int64_t *n_records) {
    yoco_status st = check_cfg(cfg);
    if (st != YOCO_OK) return st;
    if (!n_records || cap < 0 || (cap > 0 && !records) || B < 0 || n_cta < 0) return YOCO_ERR_INVALID;
    const int sms = n_cta > 0 ? n_cta : device_sm_count();
    int64_t n = 0;
    auto put = [&](int64_t a, int64_t b, int64_t c, int64_t d, int64_t e, int64_t f) {
        if (n < cap) {
            int64_t *r = records + 6 * n;
            r[0] = a; r[1] = b; r[2] = c; r[3] = d; r[4] = e; r[5] = f;
        }
        ++n;
    };
    if (kind == YOCO_SCHEDULE_PREFILL) {
        if (Tq < 0 || Tkv < 0 || q_pos0 < 0 || q_pos0 + Tq > Tkv || window < 0) return YOCO_ERR_INVALID;
        sched::PrefillShape s;
        s.B = B; s.Hq = cfg->Hq; s.Hkv = cfg->Hkv;
        s.Tq = Tq; s.Tkv = Tkv; s.q_pos0 = q_pos0; s.window = window;
        // the kernel run_prefill picks for bf16: two heads per work tile when
        // the group size is even, else one
        const bool pairs = cfg->dtype == YOCO_BF16 && sched::prefill_pairs_heads(cfg->Hq, cfg->Hkv);
        const int heads = pairs ? 2 : 1;
        const int64_t n_qtiles = (Tq + sched::kPrefillBM - 1) / sched::kPrefillBM;
        const int64_t n_work = n_qtiles * (cfg->Hq / heads) * B;
        if (n_work > INT32_MAX / 2) return YOCO_ERR_UNSUPPORTED;
        s.n_qtiles = (int32_t)n_qtiles;
        const int grid = (int)(n_work < sms ? n_work : sms);
        s.band = sched::prefill_band(grid, (cfg->Hq / cfg->Hkv) / heads,
                                     (int64_t)B * Tkv * cfg->Hkv * cfg->D * dtype_bytes(cfg->dtype) * 2, window);
        for (int c = 0; c < grid; ++c)
            for (int r = 0;; ++r) {
                const int w = sched::prefill_work_index(r, c, grid);
                if (w >= n_work) break;
                const sched::PrefillWork x = pairs ? sched::prefill_pair_work(s, w) : sched::prefill_work(s, w);
                for (int t = 0; t < x.n_kv; ++t)
                    for (int hh = 0; hh < heads; ++hh)
                        put(c, x.b, x.h + hh, x.qt, x.jt_lo + t, sched::prefill_tile_masked(s, x, t) ? 1 : 0);
            }
    } else if (kind == YOCO_SCHEDULE_DECODE) {
        if (max_len < 1 || (B > 0 && (!seq_start || !seq_len))) return YOCO_ERR_INVALID;
        DecodePlan pl;
        if (!make_decode_plan(B, max_len, cfg->Hq, cfg->Hkv, cfg->D, cfg->dtype, &pl))
            return YOCO_ERR_UNSUPPORTED;
        // the compact unit list, sequence by sequence, as the kernel enumerates it
        // (the cache's row count is not an argument here: a sequence is in
        // range when 1 <= seq_len <= max_len and seq_start >= 0)
        auto units = [&](int b) {
            return sched::decode_seq_ok(seq_start[b], seq_len[b], max_len, INT64_MAX)
                       ? sched::decode_units(seq_len[b], pl.split, pl.n_split)
                       : 0;
        };
        int64_t total = 0;
        for (int b = 0; b < B; ++b) total += units(b);
        const int64_t slots = (int64_t)B * pl.n_split;
        const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(slots, sms));
        for (int c = 0; c < grid; ++c) {
            int b = 0;
            int64_t before = 0;  // units of sequences < b
            for (int64_t u = c; u < total; u += grid) {
                while (before + units(b) <= u) before += units(b++);
                const int64_t sidx = u - before;
                const int64_t t0 = sidx * pl.split;
                const int64_t n_tok = std::min<int64_t>(pl.split, seq_len[b] - t0);
                put(c, b, sidx, seq_start[b] + t0, n_tok, (n_tok + pl.stage_tokens - 1) / pl.stage_tokens);
            }
        }
    } else {
        return YOCO_ERR_INVALID;
    }
    *n_records = n;
    return YOCO_OK;
}

double yoco_cache_bytes(int32_t L_self, int32_t window, int64_t N, const yoco_attn_cfg *cfg) {
    if (!cfg || L_self < 0 || window < 0 || N < 0 || cfg->Hkv < 1 || cfg->D < 1) return -1.0;
    const double row = 2.0 * cfg->Hkv * cfg->D * (cfg->dtype == YOCO_BF16 ? 2.0 : 4.0);
    const int64_t c = window < N ? window : N;
    return row * ((double)N + (double)L_self * (double)c);
}

yoco_status yoco_debug_wait_timeout_probe(cudaStream_t stream) {
    return from_cuda(launch_wait_timeout_probe(stream));
}

yoco_status yoco_get_device_status(cudaStream_t stream) {
    const cudaError_t e = cudaStreamSynchronize(stream);
    const unsigned int s = read_and_clear_status_decode() | read_and_clear_status_prefill_tc() |
                           read_and_clear_status_prefill_pair() | read_and_clear_status_project_tc() |
                           read_and_clear_status_gret_tc() | read_and_clear_status_linear() |
                           read_and_clear_status_ring() | read_and_clear_status_step_proj() |
                           read_and_clear_status_tree() | read_and_clear_status_tree_tc() |
                           read_and_clear_status_commit();
    if (s & 1u) return YOCO_ERR_TIMEOUT;
    if (s & 2u) return YOCO_ERR_INVALID;
    return e == cudaSuccess ? YOCO_OK : YOCO_ERR_CUDA;
}

}  // extern "C"
