"""Rotary positions and their gradient against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import workloads as wl
from tests import tree_ref as tr

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="by_parts", factor=16.0, orig_len=4096)]


def assert_rotated(got, x, pos, w, m, rot, layout, dtype, backward=False):
    """Per element of a pair (a, b): fp32 sine and cosine, off by 2 ulp of 1 and
    by the fraction of a turn's rounding, 2^-25 turns = 2 pi 2^-25; two products
    and a sum, 2^-24 each; in all below 2^-21 (|a| + |b|) m.  The angle itself,
    formed in 64 bits from rounded frequencies, is off by 4 2^-53 |t|.  One
    rounding to the output's type."""
    ref = tr.rope(x, pos, w, m, rot, layout, backward)
    y = tr.f64(x)
    ia = np.arange(rot // 2) if layout == "half" else 2 * np.arange(rot // 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    tol = np.zeros_like(ref)
    size = m * (np.abs(y[..., ia]) + np.abs(y[..., ib]))
    far = 2.0 ** -51 * np.abs(np.asarray(pos, np.float64))[..., None, None] * w
    tol[..., ia] = tol[..., ib] = size * (2.0 ** -21 + far)
    tol += np.abs(ref) * torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -7)
    tol[..., rot:] = 0
    bad = ~(np.abs(tr.f64(got) - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} elements off, first at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 64), (128, 48), (128, 128)])
@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 4, 2), (3, 37, 8, 1), (2, 1500, 4, 4)])
def test_rope(cuda_lib, dtype, layout, D, rot, B, T, Hq, Hkv):
    q, k = wl.normal((B, T, Hq, D), 2000, dtype), wl.normal((B, T, Hkv, D), 2001, dtype)
    pos = wl.randint_inclusive((B, T), 2002, 0, 1 << 20)
    for i, sc in enumerate(SCALINGS):
        cfg = cuda_lib.rope_config(rot, theta=640000.0, layout=layout, **sc)
        w, m = tr.inv_freq(rot, 640000.0, **sc)
        back = bool(i & 1)
        qo, ko = cuda_lib.rope(q.cuda(), k.cuda(), cfg, pos=pos.cuda(), backward=back)
        assert_rotated(qo, q, pos, w, m, rot, layout, dtype, back)
        assert_rotated(ko, k, pos, w, m, rot, layout, dtype, back)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_one_input_and_default_positions(cuda_lib, dtype, layout):
    B, T, Hq, Hkv, D, rot = 2, 21, 6, 3, 64, 32
    q, k = wl.normal((B, T, Hq, D), 2010, dtype), wl.normal((B, T, Hkv, D), 2011, dtype)
    cfg = cuda_lib.rope_config(rot, layout=layout)
    w, m = tr.inv_freq(rot)
    pos = (torch.arange(T) + 1000).expand(B, T)
    qd, kd = q.cuda(), k.cuda()
    qo, none = cuda_lib.rope(qd, None, cfg, pos0=1000)
    assert none is None
    assert_rotated(qo, q, pos, w, m, rot, layout, dtype)
    none, ko = cuda_lib.rope(None, kd, cfg, pos0=1000)
    assert none is None
    assert_rotated(ko, k, pos, w, m, rot, layout, dtype)
    a, b = cuda_lib.rope(qd, kd, cfg, pos0=1000, q_out=qd, k_out=kd)
    assert a is qd and b is kd
    assert torch.equal(qd, qo) and torch.equal(kd, ko)
    # one token a sequence, without a time axis
    p = torch.tensor([5, 70000])
    qo, ko = cuda_lib.rope(q[:, 0].contiguous().cuda(), k[:, 0].contiguous().cuda(), cfg, pos=p.cuda())
    assert_rotated(qo, q[:, 0], p, w, m, rot, layout, dtype)
    assert_rotated(ko, k[:, 0], p, w, m, rot, layout, dtype)


def test_extreme_positions(cuda_lib):
    D = rot = 128
    pos = torch.tensor([[0, 1, -1, -123457, 2 ** 31, 2 ** 40 + 1, 2 ** 52 - 1]])
    q = wl.normal((1, 7, 2, D), 2020, FP)
    cfg = cuda_lib.rope_config(rot)
    qo, _ = cuda_lib.rope(q.cuda(), None, cfg, pos=pos.cuda())
    assert torch.equal(qo[0, 0].cpu(), q[0, 0])
    # the reference's own argument reduction is exact; its product is one rounding, within the bound
    assert_rotated(qo[:, :5], q[:, :5], pos[:, :5], *tr.inv_freq(rot), rot, "half", FP)
    assert torch.isfinite(qo).all()
    # lengths of pairs stay, whatever the angle: sin and cos within 2^-21 each
    a, b = qo[..., :64].double(), qo[..., 64:].double()
    x, y = q[..., :64].double().cuda(), q[..., 64:].double().cuda()
    assert torch.all(((a * a + b * b).sqrt() - (x * x + y * y).sqrt()).abs() <= 2.0 ** -20 * (x.abs() + y.abs()))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient(cuda_lib, layout):
    """backward is the transpose of the forward map, and agrees with differences."""
    B, T, H, D, rot = 2, 9, 4, 64, 48
    cfg = cuda_lib.rope_config(rot, layout=layout, scaling="by_parts", factor=4.0, orig_len=64)
    x, g = wl.normal((B, T, H, D), 2030, FP).cuda(), wl.normal((B, T, H, D), 2031, FP).cuda()
    pos = wl.randint_inclusive((B, T), 2032, 0, 5000).cuda()
    f = lambda z: cuda_lib.rope(z, None, cfg, pos=pos)[0]
    dx = cuda_lib.rope(g, None, cfg, pos=pos, backward=True)[0]
    # <g, f(x)> = <f^T g, x>: both sums of the same bilinear terms, each term off
    # by at most 2^-21 of its size on either side
    size = 2 * cfg.mscale * float((g.abs().sum() * x.abs().max()).double())
    lhs, rhs = (g.double() * f(x).double()).sum(), (dx.double() * x.double()).sum()
    assert abs(float(lhs - rhs)) <= 2 * 2.0 ** -21 * size
    # f is linear: the difference quotient with step 1 along an axis is exact but for roundings
    for at in [(0, 0, 0, 0), (1, 8, 3, 47), (0, 3, 2, 23), (1, 1, 1, 24), (0, 5, 0, 63)]:
        e = torch.zeros_like(x)
        e[at] = 1
        quotient = float((g.double() * (f(x + e).double() - f(x).double())).sum())
        near = g[at[:3]].abs().max() * (x[at[:3]].abs().max() + 1)
        assert abs(quotient - float(dx[at])) <= 8 * 2.0 ** -21 * cfg.mscale * float(near)


def test_graph_and_refusals(cuda_lib):
    q, k = wl.normal((2, 5, 4, 64), 2040).cuda(), wl.normal((2, 5, 2, 64), 2041).cuda()
    cfg = cuda_lib.rope_config(64)
    pos = torch.arange(10, device="cuda").view(2, 5) * 1000
    cuda_lib.rope(q, k, cfg, pos=pos)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = cuda_lib.rope(q, k, cfg, pos=pos)
    q.mul_(2)
    pos.add_(7)
    g.replay()
    want = cuda_lib.rope(q, k, cfg, pos=pos)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    for bad in [dict(pos=pos.int()), dict(pos=pos[:1]), dict(q_out=q[:, :1]), dict(k_out=k.float())]:
        with pytest.raises(ValueError):
            cuda_lib.rope(q, k, cfg, **{"pos": pos, **bad})
    with pytest.raises(ValueError):
        cuda_lib.rope(None, None, cfg)
    with pytest.raises(ValueError):
        cuda_lib.rope(q, None, cfg, k_out=k)
    with pytest.raises(ValueError):
        cuda_lib.rope(q.transpose(1, 2), None, cfg)
    with pytest.raises(cuda_lib.YocoError):      # more than the head has
        cuda_lib.rope(q, k, cuda_lib.rope_config(128), pos=pos)


def test_outputs_side_by_side_and_shifted(cuda_lib):
    """Outputs that touch the inputs' buffers are taken, ones that overlap them refused."""
    T, H, D = 4, 2, 64
    buf = wl.normal((5, T, H, D), 2050).cuda()
    keep = buf.clone()
    cfg = cuda_lib.rope_config(64)
    q, k = buf[None, 1], buf[None, 3]
    want = cuda_lib.rope(q, k, cfg, pos0=9)
    cuda_lib.rope(q, k, cfg, pos0=9, q_out=buf[None, 2], k_out=buf[None, 4])
    assert torch.equal(buf[None, 2], want[0]) and torch.equal(buf[None, 4], want[1])
    assert torch.equal(buf[[0, 1, 3]], keep[[0, 1, 3]])
    flat = buf.view(1, 5 * T, H, D)
    for bad in [dict(q_out=flat[:, T + 1:2 * T + 1]), dict(q_out=k), dict(k_out=q), dict(k_out=flat[:, 3 * T - 1:4 * T - 1]),
                dict(q_out=buf[None, 0], k_out=buf[None, 0])]:
        before = buf.clone()
        with pytest.raises(cuda_lib.YocoError):
            cuda_lib.rope(q, k, cfg, pos0=9, **bad)
        assert torch.equal(buf, before)
    cuda_lib.rope(q, k, cfg, pos0=9, q_out=q, k_out=k)
    assert torch.equal(buf[None, 1], want[0]) and torch.equal(buf[None, 3], want[1])
