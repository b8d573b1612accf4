// Rotary positions of Q and K, and their gradient (sm_100a).
//
// The pages give the rotary base (theta) and no more ("You Only Cache Once",
// paperlayer summary, Appendix C); the attention kernels take Q and K that
// carry their positions already, and this is the call that puts them there.
// The first rot elements of a head are rot / 2 pairs (a, b) -- elements i and
// i + rot / 2, or 2 i and 2 i + 1 -- and pair i of a token at position p turns
// by t = p w_i:  a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t).
// The map is linear, so the gradient of (a, b) is the same turn by -t.
//
// Bound by memory: each element is read once and written once, and an angle
// serves all Hq + Hkv heads of its token.  A CTA therefore forms the sines and
// cosines of its tokens once, in shared memory, and then streams the heads
// through registers in 16-byte chunks, two in flight a thread and six CTAs an
// SM: 32768 tokens of 40 bf16 heads of 128 take 104 us, 6.45 TB/s read and
// written (98% of the measured copy); with four units in flight a thread, and
// fewer CTAs for their registers, 140 us, and with the pairs' sines in order,
// which puts the units of a head on the same banks, 121 us.  The angle is formed in 64 bits and
// reduced to a fraction of a turn before it is rounded to 32: at a position of
// one million the product itself in 32 bits would be off by 0.03 radians.
#include <cmath>

#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace yoco {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 64;
struct RopeParams {
    const void *q, *k;
    void *q_out, *k_out;
    const int64_t *pos;
    int64_t n, T, pos0;
    int32_t Hq, H;             // query heads; all heads of a token
    int32_t rot, tokens;       // tokens of a CTA
    float sin_sign, mscale;
    double turns[kMaxPairs];   // w_i / 2 pi
};

template <typename T>
YOCO_DEV uint4 pack16(const float *f);
template <>
YOCO_DEV uint4 pack16<float>(const float *f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
YOCO_DEV uint4 pack16<__nv_bfloat16>(const float *f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A unit of work is two 16-byte chunks of one head: a chunk of the a's with
// that of their b's, two chunks in a row of interleaved pairs, or two in a row
// of the part that does not turn (copied).
template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int EPC = Chunk<T>::N;
    constexpr int UNITS = D / (2 * EPC);   // a head
    // cosine and sine of pair i of a token, at [token][i % EPC][i / EPC]: the units of
    // a head read theirs from consecutive words
    extern __shared__ float2 s_cs[];
    pdl_trigger();
    pdl_wait();
    const int pairs = p.rot / 2;
    const int64_t tok0 = (int64_t)blockIdx.x * p.tokens;
    const int cnt = (int)min((int64_t)p.tokens, p.n - tok0);
    const int per_token = p.H * UNITS;
    const int total = cnt * per_token;
    const int rot_units = p.rot / (2 * EPC);
    const int stride = gridDim.y * kRopeThreads;
    uint4 x0, x1;
    int at = -1;        // the unit's first entry of s_cs, or -1: copied
    int gap = 0;        // from its first chunk to its second
    T *out = nullptr;   // null: nothing to do
    auto load = [&](int item) {
        out = nullptr;
        if (item >= total) return;
        const int t = item / per_token, rem = item - t * per_token;
        const int h = rem / UNITS, un = rem - h * UNITS;
        const bool turns = un < rot_units, paired = turns && !INTERLEAVED;
        const int e = paired ? un * EPC : un * 2 * EPC;
        gap = paired ? pairs : EPC;
        at = turns ? t * pairs + un : -1;
        const bool is_q = h < p.Hq;
        const int64_t off = is_q ? ((tok0 + t) * p.Hq + h) * D + e : ((tok0 + t) * (p.H - p.Hq) + h - p.Hq) * D + e;
        const T *src = static_cast<const T *>(is_q ? p.q : p.k) + off;
        T *o = static_cast<T *>(is_q ? p.q_out : p.k_out) + off;
        if (!turns && src == o) return;
        x0 = *reinterpret_cast<const uint4 *>(src);
        x1 = *reinterpret_cast<const uint4 *>(src + gap);
        out = o;
    };
    int item = blockIdx.y * kRopeThreads + threadIdx.x;
    load(item);   // on its way while the angles are formed
    for (int a = threadIdx.x; a < cnt * pairs; a += kRopeThreads) {
        const int t = a / pairs, i = a - t * pairs;
        const int64_t tok = tok0 + t;
        const int64_t pos = p.pos ? p.pos[tok] : p.pos0 + tok % p.T;
        const double turn = (double)pos * p.turns[i];
        float s, c;
        sincospif(2.f * (float)(turn - rint(turn)), &s, &c);
        s_cs[t * pairs + i % EPC * rot_units + i / EPC] = make_float2(p.mscale * c, p.mscale * p.sin_sign * s);
    }
    __syncthreads();
    for (; item < total; load(item += stride)) {
        if (!out) continue;
        if (at >= 0) {
            float f[2 * EPC];
            Chunk<T>::unpack(x0, f);
            Chunk<T>::unpack(x1, f + EPC);
#pragma unroll
            for (int i = 0; i < EPC; ++i) {
                float &a = INTERLEAVED ? f[2 * i] : f[i];
                float &b = INTERLEAVED ? f[2 * i + 1] : f[EPC + i];
                const float2 cs = s_cs[at + i * rot_units];
                const float a1 = a * cs.x - b * cs.y;
                b = b * cs.x + a * cs.y;
                a = a1;
            }
            x0 = pack16<T>(f);
            x1 = pack16<T>(f + EPC);
        }
        *reinterpret_cast<uint4 *>(out) = x0;
        *reinterpret_cast<uint4 *>(out + gap) = x1;
    }
}

template <typename T, int D, bool INTERLEAVED>
cudaError_t launch(const RopeArgs &a, const RopeParams &p, dim3 grid, cudaStream_t st) {
    note_launches(1);
    return launch_pdl(rope_kernel<T, D, INTERLEAVED>, grid, dim3(kRopeThreads),
                      sizeof(float2) * p.tokens * (a.rot_dim / 2), st, p);
}

template <typename T, int D>
cudaError_t launch_l(const RopeArgs &a, const RopeParams &p, dim3 grid, cudaStream_t st) {
    return a.interleaved ? launch<T, D, true>(a, p, grid, st) : launch<T, D, false>(a, p, grid, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st) {
    RopeParams p;
    p.q = a.q; p.k = a.k; p.q_out = a.q_out; p.k_out = a.k_out; p.pos = a.pos;
    p.n = a.n; p.T = a.T; p.pos0 = a.pos0;
    p.Hq = a.q ? a.Hq : 0;
    p.H = p.Hq + (a.k ? a.Hkv : 0);
    p.rot = a.rot_dim;
    p.sin_sign = a.backward ? -1.f : 1.f;
    p.mscale = a.mscale;
    constexpr double kTwoPi = 6.283185307179586476925;
    for (int i = 0; i < a.rot_dim / 2; ++i) p.turns[i] = a.inv_freq[i] / kTwoPi;
    for (int i = a.rot_dim / 2; i < kMaxPairs; ++i) p.turns[i] = 0.0;
    // four tokens a CTA share one round of angles once that still gives every
    // SM several CTAs (eight tokens: 107 us for the 104 above); fewer tokens are
    // spread over more CTAs, one token's heads over several (16 tokens: 2.0 us)
    const int sms = device_sm_count();
    p.tokens = a.n >= (int64_t)16 * sms ? 4 : 1;
    const int64_t ctas = (a.n + p.tokens - 1) / p.tokens;
    if (ctas > INT32_MAX) return cudaErrorNotSupported;
    const int units = p.tokens * p.H * (a.D / (a.dtype == kBF16 ? 16 : 8));
    const int most = (units + kRopeThreads - 1) / kRopeThreads;
    const int spread = (int)std::min<int64_t>(most, std::max<int64_t>(1, 2 * sms / ctas));
    const dim3 grid((unsigned)ctas, (unsigned)spread);
    if (a.dtype == kBF16) {
        if (a.D == 128) return launch_l<__nv_bfloat16, 128>(a, p, grid, st);
        if (a.D == 64) return launch_l<__nv_bfloat16, 64>(a, p, grid, st);
    } else {
        if (a.D == 128) return launch_l<float, 128>(a, p, grid, st);
        if (a.D == 64) return launch_l<float, 64>(a, p, grid, st);
    }
    return cudaErrorNotSupported;
}

}  // namespace yoco
