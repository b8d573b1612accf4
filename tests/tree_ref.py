"""Plain 64-bit forms of the drafted-token operators and the rotary positions
(numpy; test infrastructure only).  Unseen keys are left out by indexing, so
whatever they hold has no effect."""
import math

import numpy as np
import torch

from tests.util import BF16_REL_L2, FP32_REL_L2

# Half a step of a rounding to bf16, relative to the value.
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy() if isinstance(t, torch.Tensor) else np.asarray(t, np.float64)


def random_tree(rng, n, reach=6):
    """Parents-first random tree of n nodes: (mask rows as Python ints, depths)."""
    masks, depths = [], []
    for i in range(n):
        parent = int(rng.integers(max(-1, i - reach), i))
        masks.append((masks[parent] if parent >= 0 else 0) | (1 << i))
        depths.append(depths[parent] + 1 if parent >= 0 else 0)
    return masks, depths


def mask_tensor(rows, N):
    """[B][n] ints -> int64 tensor [B, N] with the bits of uint64."""
    out = np.zeros((len(rows), N), dtype=np.uint64)
    for b, r in enumerate(rows):
        for i, m in enumerate(r):
            out[b, i] = m
    return torch.from_numpy(out.view(np.int64))


def attend_row(q, keys, values, scale):
    """One query row over its seen keys: (o, lse, sum of weights x |v|)."""
    D = q.shape[0]
    if keys.shape[0] == 0:
        return np.zeros(D), -math.inf, np.zeros(D)
    x = keys @ q * scale
    m = x.max()
    w = np.exp(x - m)
    l = w.sum()
    return w @ values / l, m + math.log(l), w @ np.abs(values) / l


def tree_attention(q, k_nodes, v_nodes, context, node_sees, n_nodes, scale=0.0):
    """q [B, N, Hq, D].  context(b, i) -> (keys [L, Hkv, D], values) that node i
    sees; node_sees(b, i, j) truth.  Returns o [B, N, Hq, D], lse [B, Hq, N] and
    the magnitude of each output's terms (like o)."""
    q, kn, vn = f64(q), f64(k_nodes), f64(v_nodes)
    B, N, Hq, D = q.shape
    Hkv = kn.shape[2]
    scale = scale or 1 / math.sqrt(D)
    o, mag = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, D))
    lse = np.full((B, Hq, N), -math.inf)
    for b in range(B):
        for i in range(n_nodes[b]):
            ck, cv = context(b, i)
            js = [j for j in range(n_nodes[b]) if node_sees(b, i, j)]
            for h in range(Hq):
                g = h // (Hq // Hkv)
                keys = np.concatenate([ck[:, g], kn[b, js, g]])
                vals = np.concatenate([cv[:, g], vn[b, js, g]])
                o[b, i, h], lse[b, h, i], mag[b, i, h] = attend_row(q[b, i, h], keys, vals, scale)
    return o, lse, mag


def cross_tree(q, k_nodes, v_nodes, k_cache, v_cache, starts, lens, masks=None, n_nodes=None, scale=0.0):
    B, N = q.shape[:2]
    kc, vc = f64(k_cache), f64(v_cache)
    n_nodes = [N] * B if n_nodes is None else n_nodes
    return tree_attention(q, k_nodes, v_nodes,
                          lambda b, i: (kc[starts[b]:starts[b] + lens[b]], vc[starts[b]:starts[b] + lens[b]]),
                          lambda b, i, j: (masks[b][i] >> j) & 1 if masks else j <= i, n_nodes, scale)


def swa_tree(q, k_nodes, v_nodes, node_pos, ring_k, ring_v, slot_pos, window, masks=None, n_nodes=None, scale=0.0):
    B, N = q.shape[:2]
    rk, rv, sp = f64(ring_k), f64(ring_v), np.asarray(slot_pos).astype(np.int64)
    pos = np.asarray(node_pos).astype(np.int64)
    n_nodes = [N] * B if n_nodes is None else n_nodes

    def context(b, i):
        p = pos[b, i]
        seen = (sp[b] >= 0) & (sp[b] < p) & (sp[b] > p - window)
        return rk[b][seen], rv[b][seen]

    def sees(b, i, j):
        return ((masks[b][i] >> j) & 1 if masks else j <= i) and 0 <= pos[b, i] - pos[b, j] < window
    return tree_attention(q, k_nodes, v_nodes, context, sees, n_nodes, scale)


def assert_tree(o, lse, ref, dtype, what=""):
    """Elementwise bounds.  bf16: each weight rounded once (half a step of its
    term) and the output once; the fp32 arithmetic below adds: scores of D <= 128
    products of N(0, 1) inputs, scaled by 1 / sqrt(D), are off by at most
    (D + 2) 2^-24 sum|q k| / sqrt(D) < 130 * 2^-24 * 12 < 2^-13, and a weight by
    that relative to itself, in numerator and denominator: 2^-12 in all.  The
    log-sum takes the scores' 2^-13 and its own roundings, below 2^-12.
    Over all outputs together (a flat softmax makes them far smaller than their
    terms): a rounding is off by 2^-8 / sqrt(3) rms at most, the weights' ones
    and the output's are independent, so the 2-norm is off by a share of
    sqrt(2) 2^-8 / sqrt(3) = 3.2e-3 for V of random signs, held to 5e-3; fp32 to
    the suite's 2e-5."""
    ro, rl, mag = ref
    go, gl = f64(o), f64(lse)
    tol = 2.0 ** -12 * mag + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + BF16_HALF * (mag + np.abs(ro)) * (1 + 2.0 ** -7)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty), f"{what}: rows without keys"
    assert np.all(go[empty.transpose(0, 2, 1)] == 0), f"{what}: rows without keys are not 0"
    bad = ~(np.abs(go - ro) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} outputs off, first at {np.argwhere(bad)[0]}: "
                           f"{go[bad][0]} against {ro[bad][0]} (tolerance {tol[bad][0]:.3e})")
    rel = np.linalg.norm(go - ro) / max(np.linalg.norm(ro), 1e-30)
    assert rel <= (BF16_REL_L2 if dtype == torch.bfloat16 else FP32_REL_L2), f"{what}: relative 2-norm {rel:.2e}"
    assert np.all(np.abs(gl[~empty] - rl[~empty]) <= 2.0 ** -12), f"{what}: lse off by {np.abs(gl - rl)[~empty].max()}"


def inv_freq(rot, theta=10000.0, scaling="none", factor=1.0, orig_len=0, fast=32.0, slow=1.0):
    """Frequencies (radians a position) and magnitude, from the definitions."""
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    w = np.array([theta ** (-2 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "by_parts":
        g = np.clip((orig_len * w / (2 * math.pi) - slow) / (fast - slow), 0, 1)
        return g * w + (1 - g) * w / factor, 0.1 * math.log(factor) + 1
    return w, 1.0


def rope(x, pos, w, m, rot, layout, backward=False):
    """x [..., heads, D] at pos [...]."""
    y = f64(x).copy()
    t = np.asarray(pos, np.float64)[..., None, None] * w
    c, s = m * np.cos(t), (-m if backward else m) * np.sin(t)
    ia = np.arange(rot // 2) if layout == "half" else 2 * np.arange(rot // 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y
