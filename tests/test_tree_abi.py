"""Argument checks and host helpers of the rotary positions and the drafted-token
calls, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import shared_kv_decoder_b200 as yoco
from tests import tree_ref as tr

FAKE = ctypes.c_void_p(0x10000)   # 16-byte aligned, never dereferenced: validation fails first
OTHER = ctypes.c_void_p(0x20000)
MISALIGNED = ctypes.c_void_p(0x10008)


def _cfg(Hq=32, Hkv=8, D=128, dtype=0, scale=0.0):
    return ctypes.byref(yoco.AttnCfg(Hq, Hkv, D, scale, dtype))


@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("theta", [10000.0, 640000.0])
@pytest.mark.parametrize("sc", [dict(), dict(scaling="linear", factor=3.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="by_parts", factor=16.0, orig_len=4096),
                                dict(scaling="by_parts", factor=8.0, orig_len=8192, beta_fast=4.0, beta_slow=0.5)])
def test_rope_config(rot, theta, sc):
    cfg = yoco.rope_config(rot, theta=theta, layout="interleaved", **sc)
    ref = {{"beta_fast": "fast", "beta_slow": "slow"}.get(k, k): v for k, v in sc.items()}
    w, m = tr.inv_freq(rot, theta, **ref)
    assert cfg.rot_dim == rot and cfg.layout == 1
    # pow within an ulp or two and five more operations in 64 bits
    np.testing.assert_allclose(np.array(cfg.inv_freq)[:rot // 2], w, rtol=16 * 2.0 ** -53)
    assert not np.array(cfg.inv_freq)[rot // 2:].any()
    assert abs(cfg.mscale - m) <= 4 * 2.0 ** -53 * m
    assert yoco.rope_config(rot, mscale=0.5, **sc).mscale == 0.5


@pytest.mark.parametrize("bad", [dict(rot_dim=8), dict(rot_dim=40), dict(rot_dim=144), dict(theta=0.0),
                                 dict(theta=float("inf")), dict(theta=float("nan")), dict(scaling="linear", factor=0.5),
                                 dict(scaling="ntk", factor=float("nan")), dict(scaling="by_parts", factor=2.0),
                                 dict(scaling="by_parts", factor=2.0, orig_len=64, beta_fast=1.0), dict(mscale=-1.0)])
def test_rope_config_refusals(bad):
    with pytest.raises(yoco.YocoError) as e:
        yoco.rope_config(**{"rot_dim": 64, **bad})
    assert e.value.status == yoco.ERR_INVALID


def test_rope_config_names():
    with pytest.raises(ValueError):
        yoco.rope_config(64, layout="neox")
    with pytest.raises(ValueError):
        yoco.rope_config(64, scaling="yarn")


def test_rope_arguments_rejected_before_launch():
    L = yoco.load()
    good = yoco.rope_config(64)

    def call(q=FAKE, k=FAKE, B=2, T=3, pos=None, qo=FAKE, ko=FAKE, rope=good, cfg=_cfg()):
        return L.yoco_rope(q, k, B, T, pos, 0, 0, qo, ko, ctypes.byref(rope) if rope is not None else None, cfg, None)
    assert call(rope=None) == yoco.ERR_INVALID
    assert call(cfg=None) == yoco.ERR_INVALID
    assert call(cfg=_cfg(D=96)) == yoco.ERR_UNSUPPORTED
    assert call(q=None, k=None, qo=None, ko=None) == yoco.ERR_INVALID
    assert call(q=None) == yoco.ERR_INVALID                # an output without its input
    assert call(ko=None) == yoco.ERR_INVALID
    assert call(q=MISALIGNED) == yoco.ERR_INVALID
    assert call(ko=MISALIGNED) == yoco.ERR_INVALID
    assert call(pos=MISALIGNED) == yoco.ERR_INVALID
    assert call(B=-1) == yoco.ERR_INVALID
    assert call(T=-1) == yoco.ERR_INVALID
    assert call(B=2, T=1 << 62) == yoco.ERR_INVALID
    assert call(rope=yoco.rope_config(128), cfg=_cfg(D=64)) == yoco.ERR_UNSUPPORTED
    for field, value in [("rot_dim", 8), ("rot_dim", 72), ("layout", 2), ("mscale", float("nan"))]:
        r = yoco.rope_config(64)
        setattr(r, field, value)
        assert call(rope=r) == yoco.ERR_INVALID
    r = yoco.rope_config(64)
    r.inv_freq[31] = float("inf")
    assert call(rope=r) == yoco.ERR_INVALID
    assert call(B=0) == yoco.OK and call(T=0) == yoco.OK


def test_rope_outputs_in_place_or_apart():
    L = yoco.load()
    B, T, Hq, Hkv, D = 2, 5, 8, 2, 64
    at = lambda base, byte: ctypes.c_void_p(base.value + byte)
    q, k, pos, a, b = [ctypes.c_void_p(0x1000000 * i) for i in range(1, 6)]
    rope = yoco.rope_config(64)
    for dtype, size in ((0, 2), (1, 4)):
        qb, kb, pb = B * T * Hq * D * size, B * T * Hkv * D * size, 8 * B * T

        def call(qo, ko, p=pos):
            return L.yoco_rope(q, k, B, T, p, 0, 0, qo, ko, ctypes.byref(rope), _cfg(Hq, Hkv, D, dtype), None)
        for what, size_ in [(k, kb), (pos, pb), (b, kb)]:
            for byte in (0, size_ - 16, 16 - qb):
                assert call(at(what, byte), b) == yoco.ERR_INVALID
        for what, size_ in [(q, qb), (pos, pb), (a, qb)]:
            for byte in (0, size_ - 16, 16 - kb):
                assert call(a, at(what, byte)) == yoco.ERR_INVALID
        for byte in (16, qb - 16, -16, 16 - qb):
            assert call(at(q, byte), b) == yoco.ERR_INVALID
        for byte in (16, kb - 16, -16, 16 - kb):
            assert call(a, at(k, byte)) == yoco.ERR_INVALID
    # more bytes than an address has
    assert L.yoco_rope(q, k, 1 << 30, 1 << 30, None, 0, 0, a, b, ctypes.byref(rope), _cfg(), None) == yoco.ERR_UNSUPPORTED


def test_cross_decode_tree_arguments_rejected_before_launch():
    L = yoco.load()
    B, N, M, R = 4, 16, 65536, 1 << 20
    need = L.yoco_cross_decode_tree_workspace_size(B, N, M, _cfg())
    assert need > 0

    def call(q=FAKE, kn=FAKE, kc=FAKE, rows=R, ss=FAKE, sl=FAKE, mask=None, nn=None, b=B, n=N, m=M, o=FAKE, lse=None,
             ws=FAKE, wsb=need, cfg=_cfg()):
        return L.yoco_cross_decode_tree(q, kn, FAKE, kc, FAKE, rows, ss, sl, mask, nn, b, n, m, o, lse, ws, wsb, cfg, None)
    for bad in [dict(q=None), dict(kn=None), dict(kc=MISALIGNED), dict(ss=None), dict(sl=None), dict(mask=MISALIGNED),
                dict(nn=MISALIGNED), dict(o=None), dict(lse=MISALIGNED), dict(rows=0), dict(rows=1 << 31), dict(b=-1),
                dict(n=0), dict(m=-1), dict(m=1 << 31), dict(cfg=_cfg(Hq=30)), dict(cfg=_cfg(dtype=5))]:
        assert call(**bad) == yoco.ERR_INVALID, bad
    for bad in [dict(n=65), dict(cfg=_cfg(D=96)), dict(cfg=_cfg(Hq=48, Hkv=3))]:
        assert call(**bad) == yoco.ERR_UNSUPPORTED, bad
    for bad in [dict(ws=None), dict(ws=MISALIGNED), dict(wsb=need - 1)]:
        assert call(**bad) == yoco.ERR_WORKSPACE, bad
    assert call(b=0) == yoco.OK


def test_swa_decode_tree_arguments_rejected_before_launch():
    L = yoco.load()
    B, N, W = 64, 16, 1024
    need = L.yoco_swa_decode_tree_workspace_size(B, N, W, _cfg())
    assert need == L.yoco_cross_decode_tree_workspace_size(B, N, W, _cfg())

    def call(q=FAKE, pos=FAKE, mask=None, nn=None, b=B, n=N, w=W, rk=FAKE, sp=FAKE, o=FAKE, lse=None, ws=FAKE, wsb=need,
             cfg=_cfg()):
        return L.yoco_swa_decode_tree(q, FAKE, FAKE, pos, mask, nn, b, n, w, rk, FAKE, sp, o, lse, ws, wsb, cfg, None)
    for bad in [dict(q=None), dict(pos=None), dict(pos=MISALIGNED), dict(mask=MISALIGNED), dict(nn=MISALIGNED),
                dict(rk=None), dict(sp=None), dict(o=MISALIGNED), dict(lse=MISALIGNED), dict(b=-1), dict(n=0), dict(w=0)]:
        assert call(**bad) == yoco.ERR_INVALID, bad
    assert call(n=65) == yoco.ERR_UNSUPPORTED
    for bad in [dict(ws=None), dict(ws=MISALIGNED), dict(wsb=need - 1)]:
        assert call(**bad) == yoco.ERR_WORKSPACE, bad
    assert call(b=0) == yoco.OK


def test_commit_arguments_rejected_before_launch():
    L = yoco.load()

    def cross(kn=FAKE, path=FAKE, np_=FAKE, b=2, n=8, kc=FAKE, rows=100, ss=FAKE, sl=FAKE, cap=None, nl=OTHER, cfg=_cfg()):
        return L.yoco_cross_tree_commit(kn, FAKE, path, np_, b, n, kc, FAKE, rows, ss, sl, cap, nl, cfg, None)
    for bad in [dict(kn=None), dict(path=None), dict(np_=MISALIGNED), dict(b=-1), dict(n=0), dict(kc=None), dict(rows=0),
                dict(rows=1 << 31), dict(ss=None), dict(sl=None), dict(cap=MISALIGNED), dict(nl=None), dict(nl=FAKE),
                dict(cfg=None)]:
        assert cross(**bad) == yoco.ERR_INVALID, bad
    assert cross(n=65) == yoco.ERR_UNSUPPORTED
    assert cross(b=0) == yoco.OK

    def swa(kn=FAKE, pos=FAKE, path=FAKE, np_=FAKE, b=2, n=8, w=32, rk=FAKE, sp=FAKE, cfg=_cfg()):
        return L.yoco_swa_tree_commit(kn, FAKE, pos, path, np_, b, n, w, rk, FAKE, sp, cfg, None)
    for bad in [dict(kn=MISALIGNED), dict(pos=None), dict(path=None), dict(np_=None), dict(b=-1), dict(n=0), dict(w=0),
                dict(rk=None), dict(sp=None), dict(cfg=_cfg(Hq=30))]:
        assert swa(**bad) == yoco.ERR_INVALID, bad
    assert swa(n=65) == yoco.ERR_UNSUPPORTED
    assert swa(b=0) == yoco.OK


def test_commit_outputs_apart_from_what_it_reads():
    L = yoco.load()
    B, N, W = 64, 8, 32
    at = lambda base, byte: ctypes.c_void_p(base.value + byte)
    far = [ctypes.c_void_p(0x1000000 * i) for i in range(1, 9)]

    def cross(nl, cap=far[4]):
        return L.yoco_cross_tree_commit(FAKE, FAKE, far[0], far[1], B, N, FAKE, FAKE, 100, far[2], far[3], cap, nl, _cfg(),
                                        None)
    for x, size in [(far[0], 4 * B * N), (far[1], 4 * B), (far[2], 8 * B), (far[3], 4 * B), (far[4], 4 * B)]:
        for byte in (0, size - 16, 16 - 4 * B):
            assert cross(at(x, byte)) == yoco.ERR_INVALID

    def swa(sp):
        return L.yoco_swa_tree_commit(FAKE, FAKE, far[2], far[0], far[1], B, N, W, FAKE, FAKE, sp, _cfg(), None)
    for x, size in [(far[0], 4 * B * N), (far[1], 4 * B), (far[2], 8 * B * N)]:
        for byte in (0, size - 16, 16 - 4 * B * W):
            assert swa(at(x, byte)) == yoco.ERR_INVALID


def test_sizes_beyond_any_tensor():
    L = yoco.load()
    big = 2 ** 31 - 1
    for dtype in (0, 1):
        for B, N, Hq in [(big, 64, big), (big, 2, 4), (big, 64, 8)]:
            cfg = _cfg(Hq=Hq, Hkv=Hq, dtype=dtype)
            assert L.yoco_cross_decode_tree_workspace_size(B, N, big, cfg) == 0
            assert L.yoco_cross_decode_tree(FAKE, FAKE, FAKE, FAKE, FAKE, 100, FAKE, FAKE, None, None, B, N, big, FAKE, None,
                                            FAKE, 1 << 60, cfg, None) == yoco.ERR_UNSUPPORTED
        cfg = _cfg(Hq=big, Hkv=big, dtype=dtype)
        far = [ctypes.c_void_p(0x1000000 * i) for i in range(1, 6)]
        assert L.yoco_rope(FAKE, FAKE, 1, 1, None, 0, 0, FAKE, FAKE, ctypes.byref(yoco.rope_config(64)), cfg,
                           None) == yoco.ERR_UNSUPPORTED
        assert L.yoco_cross_tree_commit(FAKE, FAKE, far[0], far[1], 1, 64, FAKE, FAKE, 100, far[2], far[3], None, far[4],
                                        cfg, None) == yoco.ERR_UNSUPPORTED
        assert L.yoco_swa_tree_commit(FAKE, FAKE, far[2], far[0], far[1], 1, 64, 8, FAKE, FAKE, far[3], cfg,
                                      None) == yoco.ERR_UNSUPPORTED


def test_tree_heads_beyond_32_bit_rows():
    # a row of 2^24 heads is 2^29 16-byte chunks (fp32, D = 128); of eight times as many, 2^32
    L = yoco.load()
    for dtype in (0, 1):
        for Hq, ok in [(1 << 24, True), ((1 << 24) + 8, False), (1 << 27, False)]:
            cfg = _cfg(Hq=Hq, Hkv=Hq // 8, dtype=dtype)
            assert (L.yoco_cross_decode_tree_workspace_size(1, 1, 64, cfg) > 0) == ok
            if not ok:
                assert L.yoco_cross_decode_tree(FAKE, FAKE, FAKE, FAKE, FAKE, 100, FAKE, FAKE, None, None, 1, 1, 64, FAKE,
                                                None, FAKE, 1 << 60, cfg, None) == yoco.ERR_UNSUPPORTED
                assert L.yoco_swa_decode_tree(FAKE, FAKE, FAKE, FAKE, None, None, 1, 1, 64, FAKE, FAKE, FAKE, FAKE, None,
                                              FAKE, 1 << 60, cfg, None) == yoco.ERR_UNSUPPORTED


def test_workspace_sizes():
    sizes = [yoco.cross_decode_tree_workspace_size(B, N, M, 32, 8, 128, torch.bfloat16)
             for B, N, M in [(32, 1, 64), (1, 1, 131072), (4, 16, 65536), (16, 64, 131072)]]
    assert all(s > 0 for s in sizes)
    # few streams, none of them long: none is needed, and a call takes NULL
    assert yoco.cross_decode_tree_workspace_size(1, 1, 2048, 32, 8, 128, torch.bfloat16) == 0
    assert yoco.swa_decode_tree_workspace_size(4, 16, 1024, 32, 8, 128, torch.bfloat16) == 0
    assert yoco.cross_decode_tree_workspace_size(1, 1, 2048, 32, 8, 128, torch.float32) > 0
    for bad in [(0, 1, 64), (1, 0, 64), (1, 65, 64), (1, 1, -1)]:
        assert yoco.cross_decode_tree_workspace_size(*bad, 32, 8, 128, torch.bfloat16) == 0
    assert yoco.swa_decode_tree_workspace_size(1, 1, 0, 32, 8, 128, torch.bfloat16) == 0


def test_cpu_tensors_are_refused():
    q, k = torch.zeros(1, 2, 4, 64), torch.zeros(1, 2, 2, 64)
    with pytest.raises(ValueError):
        yoco.rope(q, k, yoco.rope_config(64))
    with pytest.raises(ValueError):
        yoco.cross_decode_tree(q, k, k, k[0], k[0], None, None, 1)
    with pytest.raises(ValueError):
        yoco.swa_decode_tree(q, k, k, None, None, None, None, 8)
    with pytest.raises(ValueError):
        yoco.cross_tree_commit(k, k, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        yoco.swa_tree_commit(k, k, None, None, None, None, None, None, 8)
