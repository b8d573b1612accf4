"""Tree attention on each way its kernels have of sharing the work -- clusters of
every size and the numbered shares, one row tile and two -- against plain 64-bit
forms."""
import math

import numpy as np
import pytest
import torch

from tests import tree_ref as tr
from tests.test_gpu_tree import cross_case, i32, i64, ring_case, run_cross, run_swa

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def status(cuda_lib):
    yield
    assert cuda_lib.device_status() == cuda_lib.OK


def cluster_size(B, N, max_len, Hq, Hkv):
    """CTAs of a cluster in the bf16 plan, 0: numbered shares."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = N * (Hq // Hkv)
    streams = B * -(-rows // (128 if rows <= 128 else 256)) * Hkv
    tiles = -(-max_len // 128) + 1
    size = 0
    for c, room in ((2, sms // 2), (4, (sms - 16) // 4), (8, (sms - 28) // 8)):
        if streams <= room and tiles <= c * (16 if streams * c * 2 >= sms else 12):
            size = c
    return size


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G", [(33, 4), (64, 8)])    # 132 rows of a KV head; 512, two row blocks
@pytest.mark.parametrize("size,B,L", [(8, 2, 6000), (4, 9, 2300), (2, 19, 1500)])
def test_clusters_of_two_row_tiles(cuda_lib, N, G, D, size, B, L):
    """A CTA's two chains leave their partials over the tiles that both have read:
    the same outputs every time, and the right ones."""
    Hkv = 1 if N * G > 256 else 2
    lens = [L - 391 * b % L for b in range(B)]
    assert cluster_size(B, N, L, Hkv * G, Hkv) == size
    assert cuda_lib.cross_decode_tree_workspace_size(B, N, L, Hkv * G, Hkv, D, BF) == 0
    q, kn, vn, kc, vc, starts = cross_case(BF, lens, N, Hkv * G, Hkv, D, 2500)
    rng = np.random.default_rng(size)
    masks = [tr.random_tree(rng, N)[0] for _ in lens]
    o, lse = run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, masks, max_len=L)
    for _ in range(50):
        o2, lse2 = run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, masks, max_len=L)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    some = [0, B // 2, B - 1]     # the 64-bit form of three sequences
    ref = tr.cross_tree(q[some], kn[some], vn[some], kc, vc, [starts[b] for b in some], [lens[b] for b in some],
                        [masks[b] for b in some])
    tr.assert_tree(o[some], lse[some], ref, BF)


def test_rows_without_a_node_of_very_many_heads(cuda_lib):
    """A token of 2^22 fp32 heads of 128 is 2^31 bytes."""
    Hq, D = 1 << 22, 128
    q = torch.zeros(1, 1, Hq, D, device="cuda")
    kn, kc = torch.zeros(1, 1, Hq // 8, D, device="cuda"), torch.zeros(1, Hq // 8, D, device="cuda")
    o = torch.ones_like(q)
    o, lse = cuda_lib.cross_decode_tree(q, kn, kn, kc, kc, torch.zeros(1, dtype=torch.int64, device="cuda"),
                                        torch.zeros(1, dtype=torch.int32, device="cuda"), 0,
                                        n_nodes=torch.zeros(1, dtype=torch.int32, device="cuda"), want_lse=True, o=o)
    assert not o.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("size,B,L", [(8, 2, 4096), (4, 30, 900), (2, 50, 700), (0, 80, 700)])
@pytest.mark.parametrize("N,D", [(1, 128), (6, 64), (32, 128)])
def test_clusters_of_one_row_tile(cuda_lib, N, D, size, B, L):
    Hq, Hkv = 4, 1
    lens = [L - 37 * b % L for b in range(B)]
    assert cluster_size(B, N, L, Hq, Hkv) == size
    assert (cuda_lib.cross_decode_tree_workspace_size(B, N, L, Hq, Hkv, D, BF) == 0) == (size > 0)
    q, kn, vn, kc, vc, starts = cross_case(BF, lens, N, Hq, Hkv, D, 2600)
    ref = tr.cross_tree(q, kn, vn, kc, vc, starts, lens)
    tr.assert_tree(*run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, max_len=L), ref, BF)


def assert_with_bad_values(o, lse, ref, dtype):
    """Infinities and NaN where the 64-bit form has them, the rest within its bounds."""
    go, (ro, rl, mag) = tr.f64(o), ref
    bad = ~np.isfinite(ro)
    assert np.array_equal(~np.isfinite(go), bad)
    assert np.array_equal(go[bad], ro[bad], equal_nan=True)
    clear = lambda x: np.where(bad, 0, x)
    tr.assert_tree(clear(go), lse, (clear(ro), rl, clear(mag)), dtype)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B", [1, 80])                 # bf16: in clusters, and dealt in shares
@pytest.mark.parametrize("N,Hq,Hkv,D", [(4, 8, 2, 128), (9, 2, 2, 64), (40, 8, 2, 128), (33, 16, 2, 64)])
def test_bad_values_in_ring_slots_that_some_nodes_see(cuda_lib, dtype, B, N, Hq, Hkv, D):
    """Node i of a chain whose positions are 17 apart sees the slots above its window's
    lower end, so a slot's bad value reaches the first nodes and no other."""
    W, step = 1000, 17
    filled = [1500 + 13 * b for b in range(B)]
    q, kn, vn, rk, rv, sp = ring_case(dtype, B, N, W, filled, Hq, Hkv, D, 2700)
    assert (cluster_size(B, N, W, Hq, Hkv) > 0) == (B == 1)
    pos = [[f + step * i for i in range(N)] for f in filled]
    rng = np.random.default_rng(N)
    for b, f in enumerate(filled):
        for bad in (math.inf, -math.inf, math.nan, math.inf):
            last = int(rng.integers(0, N))             # the last node that sees the slot
            s = f + step * last - W + 1
            slot, g, d = s % W, int(rng.integers(0, Hkv)), int(rng.integers(0, D))
            assert f - W <= s < f and sp[b, slot] == s
            rv[b, slot, g, d] = bad
        old = (f - W) % W                              # the oldest slot, which no node sees
        assert sp[b, old] == f - W
        rv[b, old], rk[b, old] = math.nan, math.inf
        vn[b, N - 1, 0, 1] = math.inf                  # and a node that only itself sees
    o, lse = run_swa(cuda_lib, q, kn, vn, pos, rk, rv, sp, W)
    o2, lse2 = run_swa(cuda_lib, q, kn, vn, pos, rk, rv, sp, W)
    assert torch.equal(o.isnan(), o2.isnan()) and torch.equal(o.nan_to_num(), o2.nan_to_num()) and torch.equal(lse, lse2)
    some = sorted({0, B // 3, B - 1})
    with np.errstate(invalid="ignore"):
        ref = tr.swa_tree(q[some], kn[some], vn[some], [pos[b] for b in some], rk[some], rv[some], sp[some], W)
    assert not np.isfinite(ref[0]).all()
    assert_with_bad_values(o[some], lse[some], ref, dtype)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("most", [512, 1 << 20])       # bf16: in clusters, and in shares
@pytest.mark.parametrize("N", [5, 40])
def test_output_at_16_bytes_and_without_lse(cuda_lib, dtype, most, N):
    lens, Hq, Hkv, D = [300, 64, 0], 8, 2, 128
    q, kn, vn, kc, vc, starts = cross_case(dtype, lens, N, Hq, Hkv, D, 2800)
    args = [t.cuda() for t in (q, kn, vn, kc, vc)] + [i64(starts), i32(lens), most]
    nodes = i32([N, N - 1, N])
    o, lse = cuda_lib.cross_decode_tree(*args, n_nodes=nodes, want_lse=True)
    assert o.data_ptr() % 32 == 0
    tr.assert_tree(o, lse, tr.cross_tree(q, kn, vn, kc, vc, starts, lens, None, [N, N - 1, N]), dtype)
    assert torch.equal(cuda_lib.cross_decode_tree(*args, n_nodes=nodes), o)
    pad = 16 // q.element_size()
    buf = torch.full((q.numel() + 2 * pad,), 7.0, dtype=dtype, device="cuda")
    at = buf[pad:-pad].view(q.shape)
    assert at.data_ptr() % 32 == 16
    cuda_lib.cross_decode_tree(*args, n_nodes=nodes, o=at)
    assert torch.equal(at, o) and (buf[:pad] == 7).all() and (buf[-pad:] == 7).all()
    W = 300
    q, kn, vn, rk, rv, sp = ring_case(dtype, 3, N, W, [200, 1000, 0], Hq, Hkv, D, 2900)
    pos = i64([[f + i for i in range(N)] for f in (200, 1000, 0)])
    args = [t.cuda() for t in (q, kn, vn)] + [pos, rk.cuda(), rv.cuda(), torch.from_numpy(sp).cuda(), W]
    o, lse = cuda_lib.swa_decode_tree(*args, n_nodes=nodes, want_lse=True)
    assert torch.equal(cuda_lib.swa_decode_tree(*args, n_nodes=nodes), o)
    buf.fill_(7.0)
    cuda_lib.swa_decode_tree(*args, n_nodes=nodes, o=at)
    assert torch.equal(at, o) and (buf[:pad] == 7).all() and (buf[-pad:] == 7).all()
