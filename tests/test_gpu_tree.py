"""Drafted tokens: tree attention over the shared cache and over the ring, and
the commits, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import workloads as wl
from tests import tree_ref as tr

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def status(cuda_lib):
    yield
    assert cuda_lib.device_status() == cuda_lib.OK


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def i64(x):
    return torch.tensor(x, dtype=torch.int64, device="cuda")


def cross_case(dtype, lens, N, Hq, Hkv, D, seed, gap=3, fill=math.nan):
    """A packed cache whose rows between and behind the sequences hold `fill`."""
    starts, rows = [], gap
    for n in lens:
        starts.append(rows)
        rows += n + gap
    kc, vc = (torch.full((rows, Hkv, D), fill, dtype=dtype) for _ in range(2))
    for b, (s, n) in enumerate(zip(starts, lens)):
        kc[s:s + n] = wl.normal((n, Hkv, D), seed + 10 * b, dtype) if n else kc[s:s]
        vc[s:s + n] = wl.normal((n, Hkv, D), seed + 10 * b + 1, dtype) if n else vc[s:s]
    B = len(lens)
    q = wl.normal((B, N, Hq, D), seed + 5000, dtype)
    kn, vn = wl.normal((B, N, Hkv, D), seed + 5001, dtype), wl.normal((B, N, Hkv, D), seed + 5002, dtype)
    return q, kn, vn, kc, vc, starts


def run_cross(lib, q, kn, vn, kc, vc, starts, lens, masks=None, n_nodes=None, max_len=None, **kw):
    return lib.cross_decode_tree(q.cuda(), kn.cuda(), vn.cuda(), kc.cuda(), vc.cuda(), i64(starts), i32(lens),
                                 max(lens) if max_len is None else max_len,
                                 tree_mask=None if masks is None else tr.mask_tensor(masks, q.shape[1]).cuda(),
                                 n_nodes=None if n_nodes is None else i32(n_nodes), want_lse=True, **kw)


SHAPES = [(4, 2, 64), (8, 8, 64), (8, 2, 128), (8, 1, 128), (4, 4, 128)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("most", [1024, 1 << 20])    # bf16: clusters of CTAs where they fit; shares and the join
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("N,lens", [(1, [0, 1, 2, 63, 64, 65]), (3, [127, 128, 129]), (17, [300, 0, 1]),
                                    (40, [255]), (64, [1, 700])])
def test_cross_tree(cuda_lib, dtype, most, Hq, Hkv, D, N, lens):
    q, kn, vn, kc, vc, starts = cross_case(dtype, lens, N, Hq, Hkv, D, 100)
    rng = np.random.default_rng(N)
    masks = [tr.random_tree(rng, N)[0] for _ in lens]
    n_nodes = [N] + [int(rng.integers(0, N + 1)) for _ in lens[1:]]
    ref = tr.cross_tree(q, kn, vn, kc, vc, starts, lens, masks, n_nodes)
    tr.assert_tree(*run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, masks, n_nodes, most), ref, dtype, "tree")
    ref = tr.cross_tree(q, kn, vn, kc, vc, starts, lens, scale=0.3)
    tr.assert_tree(*run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, max_len=most, scale=0.3), ref, dtype, "chain")


@pytest.mark.parametrize("dtype", [BF, FP])
def test_cross_tree_long_and_shared_between_ctas(cuda_lib, dtype):
    # more tiles than CTAs, lengths that cut streams anywhere, more than 32 sequences
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 900, 37)] + [5003]
    N = 5
    q, kn, vn, kc, vc, starts = cross_case(dtype, lens, N, 8, 2, 128, 300, gap=0)
    masks = [tr.random_tree(rng, N)[0] for _ in lens]
    n_nodes = [int(x) for x in rng.integers(0, N + 1, len(lens))]
    ref = tr.cross_tree(q, kn, vn, kc, vc, starts, lens, masks, n_nodes)
    tr.assert_tree(*run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, masks, n_nodes, max_len=8192), ref, dtype)


@pytest.mark.parametrize("N,Hq,Hkv,D,lens", [(3, 32, 8, 128, [3255, 6355, 4000, 5121, 3968, 4097, 6000]),
                                             (2, 16, 2, 128, [20001, 9000, 12345]), (11, 4, 4, 128, [15000, 1, 8191, 130]),
                                             (30, 16, 2, 128, [4500, 7000])])
def test_cross_tree_many_tiles_a_segment(cuda_lib, N, Hq, Hkv, D, lens):
    """Segments of dozens of tiles that start and end anywhere, where V tiles are
    loaded while others are still in use."""
    q, kn, vn, kc, vc, starts = cross_case(BF, lens, N, Hq, Hkv, D, 350)
    rng = np.random.default_rng(N)
    masks = [tr.random_tree(rng, N)[0] for _ in lens]
    ref = tr.cross_tree(q, kn, vn, kc, vc, starts, lens, masks)
    for _ in range(3):
        tr.assert_tree(*run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, masks), ref, BF)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("most", [128, 1 << 20])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(6, 4, 2, 64), (64, 8, 2, 128)])
def test_rows_that_see_nothing(cuda_lib, dtype, most, N, Hq, Hkv, D):
    lens = [0, 0, 5]
    q, kn, vn, kc, vc, starts = cross_case(dtype, lens, N, Hq, Hkv, D, 400)
    masks = [[0] * N, [(1 << i) if i % 3 else 0 for i in range(N)], [0] * N]
    ref = tr.cross_tree(q, kn, vn, kc, vc, starts, lens, masks)
    assert np.isneginf(ref[1][0]).all()
    tr.assert_tree(*run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, masks, max_len=most), ref, dtype)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("most", [128, 1 << 20])
def test_no_nodes_at_all(cuda_lib, dtype, most):
    lens = [100, 0]
    q, kn, vn, kc, vc, starts = cross_case(dtype, lens, 3, 4, 2, 64, 450)
    o, lse = run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, None, [0, 0], max_len=most)
    assert not o.any() and torch.isneginf(lse).all()
    q, kn, vn, rk, rv, sp = ring_case(dtype, 2, 3, 40, [5, 90], 4, 2, 64, 460)
    o, lse = run_swa(cuda_lib, q, kn, vn, [[5, 6, 7], [90, 91, 92]], rk, rv, sp, 40, None, [0, 0])
    assert not o.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("B,L", [(2, 4096), (14, 300), (30, 900)])
def test_clusters_of_every_size(cuda_lib, B, L):
    """Streams for clusters of eight, four and two CTAs."""
    Hq, Hkv, D, N = 4, 1, 128, 6
    lens = [L - 37 * b % L for b in range(B)]
    assert cuda_lib.cross_decode_tree_workspace_size(B, N, L, Hq, Hkv, D, BF) == 0
    q, kn, vn, kc, vc, starts = cross_case(BF, lens, N, Hq, Hkv, D, 470)
    ref = tr.cross_tree(q, kn, vn, kc, vc, starts, lens)
    tr.assert_tree(*run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, max_len=L), ref, BF)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("most", [256, 1 << 20])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(5, 4, 2, 64), (40, 8, 2, 128)])
def test_unseen_nodes_may_hold_anything_and_seen_ones_count(cuda_lib, dtype, most, bad, N, Hq, Hkv, D):
    lens = [130, 64]
    q, kn, vn, kc, vc, starts = cross_case(dtype, lens, N, Hq, Hkv, D, 500)
    # node 2's K and V are bad; only node 4 sees it, whose rows have to show it
    masks = [[((1 << (i + 1)) - 1) & ~(1 << 2) for i in range(N)] for _ in lens]
    masks[0][4] |= 1 << 2
    kn[0, 2], vn[0, 2] = bad, bad
    vn[1, 2, :, 7] = bad                       # one element of V, seen by node 3 of sequence 1
    masks[1][3] |= 1 << 2
    o, lse = run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, masks, max_len=most)
    go = tr.f64(o)
    assert not np.isfinite(go[0, 4]).any()
    assert not np.isfinite(go[1, 3, :, 7]).any()
    if math.isinf(bad):
        assert np.array_equal(go[1, 3, :, 7], np.full(Hq, bad))
    clean = [m[:] for m in masks]
    clean[0][4] &= ~(1 << 2)
    clean[1][3] &= ~(1 << 2)
    kn2, vn2 = kn.clone(), vn.clone()
    kn2[0, 2], vn2[0, 2], vn2[1, 2] = 0, 0, 0
    ref = tr.cross_tree(q, kn2, vn2, kc, vc, starts, lens, clean)
    rows = np.ones((2, N), bool)
    rows[0, 4] = rows[1, 3] = False
    assert np.isfinite(go[rows]).all()
    tol = 2.0 ** -12 * ref[2] + 1e-30
    if dtype == BF:
        tol = tol + tr.BF16_HALF * (ref[2] + np.abs(ref[0])) * (1 + 2.0 ** -7)
    assert np.all(np.abs(go[rows] - ref[0][rows]) <= tol[rows])
    # the other columns of the row with one bad element of V: as if it were finite
    vn3 = vn.clone()
    vn3[1, 2, :, 7] = 0
    one = [m[:] for m in masks]
    ref1 = tr.cross_tree(q[1:], kn[1:], vn3[1:], kc, vc, starts[1:], lens[1:], one[1:])
    cols = [d for d in range(D) if d != 7]
    t1 = 2.0 ** -12 * ref1[2] + (tr.BF16_HALF * (ref1[2] + np.abs(ref1[0])) * (1 + 2.0 ** -7) if dtype == BF else 0)
    assert np.all(np.abs(go[1, 3][:, cols] - ref1[0][0, 3][:, cols]) <= t1[0, 3][:, cols])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("most", [128, 1 << 20])
def test_nan_in_q_stays_in_its_row(cuda_lib, dtype, most):
    lens, N = [70], 4
    q, kn, vn, kc, vc, starts = cross_case(dtype, lens, N, 4, 2, 64, 550)
    q[0, 1, 2, 3] = math.nan
    o, lse = run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, max_len=most)
    go, gl = tr.f64(o), tr.f64(lse)
    assert np.isnan(go[0, 1, 2]).all() and np.isnan(gl[0, 2, 1])
    go[0, 1, 2], gl[0, 2, 1] = 0, 0
    assert np.isfinite(go).all() and np.isfinite(gl).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("many", [1, 40])            # bf16: in clusters, and dealt in shares
def test_sequences_out_of_range(cuda_lib, dtype, many):
    lens, N = [40, 33, 20, 64, 10, 12], 3
    q, kn, vn, kc, vc, starts = cross_case(dtype, lens, N, 4, 2, 64, 600)
    given, at, nodes = list(lens), list(starts), [N] * 6
    given[1] = 65                 # above max_len
    given[2] = -1
    at[3] = kc.shape[0] - 63      # runs past the cache
    nodes[4] = N + 1
    at[5] = -1
    rep = lambda t: t.repeat(many, 1, 1, 1)
    o, lse = run_cross(cuda_lib, rep(q), rep(kn), rep(vn), kc, vc, at * many, given * many, None, nodes * many, max_len=64)
    assert cuda_lib.device_status() == cuda_lib.ERR_INVALID
    # (copies are not equal to the bit: shares cut each one's tiles elsewhere)
    ref = tr.cross_tree(q, kn, vn, kc, vc, starts, lens, None, [N, 0, 0, 0, 0, 0])
    for i in range(0, 6 * many, 6):
        tr.assert_tree(o[i:i + 6], lse[i:i + 6], ref, dtype)


def ring_case(dtype, B, N, W, filled, Hq, Hkv, D, seed, empty=math.nan):
    """Rings that hold the newest positions below filled[b]; empty slots hold `empty`."""
    rk, rv = wl.normal((B, W, Hkv, D), seed, dtype), wl.normal((B, W, Hkv, D), seed + 1, dtype)
    sp = np.full((B, W), -1, np.int32)
    for b in range(B):
        for p in range(max(0, filled[b] - W), filled[b]):
            sp[b, p % W] = p
        free = torch.from_numpy(sp[b] < 0)
        rk[b, free], rv[b, free] = empty, empty
    q = wl.normal((B, N, Hq, D), seed + 2, dtype)
    kn, vn = wl.normal((B, N, Hkv, D), seed + 3, dtype), wl.normal((B, N, Hkv, D), seed + 4, dtype)
    return q, kn, vn, rk, rv, sp


def run_swa(lib, q, kn, vn, pos, rk, rv, sp, W, masks=None, n_nodes=None, **kw):
    return lib.swa_decode_tree(q.cuda(), kn.cuda(), vn.cuda(), i64(np.asarray(pos).tolist()), rk.cuda(), rv.cuda(),
                               torch.from_numpy(sp).cuda(), W,
                               tree_mask=None if masks is None else tr.mask_tensor(masks, q.shape[1]).cuda(),
                               n_nodes=None if n_nodes is None else i32(n_nodes), want_lse=True, **kw)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("W,N,filled", [(1, 4, [0, 3]), (5, 9, [2, 100]), (32, 7, [272, 0, 31]), (128, 1, [127, 128, 129]),
                                        (200, 33, [1000]), (300, 64, [299, 70000])])
def test_swa_tree(cuda_lib, dtype, Hq, Hkv, D, W, N, filled):
    B = len(filled)
    q, kn, vn, rk, rv, sp = ring_case(dtype, B, N, W, filled, Hq, Hkv, D, 700)
    rng = np.random.default_rng(W + N)
    trees = [tr.random_tree(rng, N) for _ in filled]
    masks, pos = [t[0] for t in trees], [[f + d for d in t[1]] for f, t in zip(filled, trees)]
    n_nodes = [N] + [int(rng.integers(0, N + 1)) for _ in filled[1:]]
    ref = tr.swa_tree(q, kn, vn, pos, rk, rv, sp, W, masks, n_nodes)
    tr.assert_tree(*run_swa(cuda_lib, q, kn, vn, pos, rk, rv, sp, W, masks, n_nodes), ref, dtype, "tree")
    pos = [[f + i for i in range(N)] for f in filled]   # a chain, longer than the window where N > W
    ref = tr.swa_tree(q, kn, vn, pos, rk, rv, sp, W)
    tr.assert_tree(*run_swa(cuda_lib, q, kn, vn, pos, rk, rv, sp, W), ref, dtype, "chain")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(5, 8, 2, 128), (40, 16, 4, 64)])
def test_swa_tree_many_sequences(cuda_lib, dtype, N, Hq, Hkv, D):
    """More streams than SMs: shares that start and end anywhere."""
    B, W = 45, 300
    rng = np.random.default_rng(9)
    filled = [int(x) for x in rng.integers(0, 2 * W, B)]
    q, kn, vn, rk, rv, sp = ring_case(dtype, B, N, W, filled, Hq, Hkv, D, 750)
    trees = [tr.random_tree(rng, N) for _ in filled]
    masks, pos = [t[0] for t in trees], [[f + d for d in t[1]] for f, t in zip(filled, trees)]
    n_nodes = [int(x) for x in rng.integers(0, N + 1, B)]
    ref = tr.swa_tree(q, kn, vn, pos, rk, rv, sp, W, masks, n_nodes)
    tr.assert_tree(*run_swa(cuda_lib, q, kn, vn, pos, rk, rv, sp, W, masks, n_nodes), ref, dtype)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_swa_tree_odd_rings(cuda_lib, dtype):
    # slots in no order, positions ahead of the nodes', empty ones with infinities, nodes in any order
    W, N, B = 260, 6, 3
    q, kn, vn, rk, rv, sp = ring_case(dtype, B, N, W, [400, 400, 400], 8, 2, 128, 800)
    rng = np.random.default_rng(3)
    sp[0] = rng.permutation(sp[0])
    sp[1, ::7] = 1000
    sp[2, 3::5] = -1
    rv[2, 3::5] = math.inf
    sp[0, 5] = -(1 << 31)
    rk[0, 5] = math.nan
    rv[0, 5] = math.nan
    pos = [[405, 400, 399, 0, 2 ** 31 + 5, -7], [400 + i for i in range(N)], [650, 600, 401, 640, 400, 402]]
    masks = [[(1 << N) - 1] * N, [1 << i for i in range(N)], [(1 << N) - 1] * N]
    ref = tr.swa_tree(q, kn, vn, pos, rk, rv, sp, W, masks)
    tr.assert_tree(*run_swa(cuda_lib, q, kn, vn, pos, rk, rv, sp, W, masks), ref, dtype)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_swa_tree_bad_value_in_a_seen_slot(cuda_lib, dtype):
    W, N, B = 256, 4, 1
    q, kn, vn, rk, rv, sp = ring_case(dtype, B, N, W, [300], 8, 2, 128, 850)
    pos = [[300, 301, 302, 303]]
    # position 46 is in the window of nodes 0 and 1 only (46 > p - 256)
    slot = 46 % W
    sp[0, slot] = 46
    rv[0, slot, 1, 5] = math.inf
    o, lse = run_swa(cuda_lib, q, kn, vn, pos, rk, rv, sp, W)
    go = tr.f64(o)
    assert np.array_equal(go[0, :2, 4:, 5], np.full((2, 4), math.inf))
    rv[0, slot, 1, 5] = 0
    ref = tr.swa_tree(q, kn, vn, pos, rk, rv, sp, W)
    assert np.isfinite(go[0, 2:]).all() and np.isfinite(go[0, :, :4]).all()
    go[0, :2, 4:, 5] = ref[0][0, :2, 4:, 5]
    tr.assert_tree(go, lse, ref, dtype)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_one_node_is_the_decode_step(cuda_lib, dtype):
    """A chain of one node equals yoco_cross_decode with the node appended, and
    yoco_swa_decode with it as the new token."""
    lens, Hq, Hkv, D = [77, 300], 8, 2, 128
    q, kn, vn, kc, vc, starts = cross_case(dtype, lens, 1, Hq, Hkv, D, 900, gap=1, fill=0.0)
    o, lse = run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens)
    new_len = cuda_lib.cross_tree_commit(kn.cuda(), vn.cuda(), i32([[0], [0]]), i32([1, 1]), kd := kc.cuda(),
                                         vd := vc.cuda(), i64(starts), i32(lens))
    assert new_len.tolist() == [78, 301]
    od, ld = cuda_lib.cross_decode(q[:, 0].contiguous().cuda(), kd, vd, i64(starts), new_len, 301, want_lse=True)
    ref = tr.cross_tree(q, kn, vn, kc, vc, starts, lens)
    tr.assert_tree(o, lse, ref, dtype)
    tr.assert_tree(od[:, None], ld[:, :, None], ref, dtype)
    W = 32
    q, kn, vn, rk, rv, sp = ring_case(dtype, 2, 1, W, [50, 3], Hq, Hkv, D, 950, empty=0.0)
    pos = [[50], [3]]
    o, lse = run_swa(cuda_lib, q, kn, vn, pos, rk, rv, sp, W)
    ref = tr.swa_tree(q, kn, vn, pos, rk, rv, sp, W)
    tr.assert_tree(o, lse, ref, dtype)
    ring = rk.cuda(), rv.cuda(), torch.from_numpy(sp).cuda()
    mine = [t.clone() for t in ring]
    od = cuda_lib.swa_decode(q[:, 0].contiguous().cuda(), kn[:, 0].contiguous().cuda(), vn[:, 0].contiguous().cuda(),
                             i64([50, 3]), *ring, W)
    tr.assert_tree(od[:, None], lse, ref, dtype)
    cuda_lib.swa_tree_commit(kn.cuda(), vn.cuda(), i64(pos), i32([[0], [0]]), i32([1, 1]), *mine, W)
    for a, b in zip(mine, ring):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_cross_commit(cuda_lib, dtype):
    N, Hkv, D = 9, 2, 64
    lens = [0, 5, 64, 7, 8, 3, 2, 30]
    q, kn, vn, kc, vc, starts = cross_case(dtype, lens, N, 4, Hkv, D, 1000, gap=N, fill=0.5)
    path = [[0, 3, 8] + [0] * 6, [2] + [-5] * 8, [99] * 9, [0, 9] + [0] * 7, [0] * 9, [1, 1, 4] + [0] * 6,
            [0, 1, 2, 3] + [0] * 5, list(range(9))]
    n_path = [3, 1, 0, 2, 10, 3, 4, 9]
    cap = [n + N for n in lens]
    cap[6] = lens[6] + 3                                 # no room for four
    kd, vd, new_len = kc.cuda(), vc.cuda(), i32([-1] * 8)
    got = cuda_lib.cross_tree_commit(kn.cuda(), vn.cuda(), i32(path), i32(n_path), kd, vd, i64(starts), i32(lens),
                                     seq_cap=i32(cap), new_len=new_len)
    assert cuda_lib.device_status() == cuda_lib.ERR_INVALID
    assert got is new_len
    wk, wv, want = kc.clone(), vc.clone(), list(lens)
    for b in (0, 1, 2, 5, 7):
        for j in range(n_path[b]):
            wk[starts[b] + lens[b] + j] = kn[b, path[b][j]]
            wv[starts[b] + lens[b] + j] = vn[b, path[b][j]]
        want[b] += n_path[b]
    assert torch.equal(kd.cpu(), wk) and torch.equal(vd.cpu(), wv) and new_len.tolist() == want
    # without caps the cache's end is the bound
    at = i64([kc.shape[0] - 5])
    for n, ok in ((5, True), (6, False)):
        r = cuda_lib.cross_tree_commit(kn[:1].cuda(), vn[:1].cuda(), i32([list(range(9))]), i32([n]), kd, vd, at, i32([0]))
        assert r.tolist() == [n if ok else 0]
        assert cuda_lib.device_status() == (cuda_lib.OK if ok else cuda_lib.ERR_INVALID)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("W", [1, 4, 32])
def test_swa_commit(cuda_lib, dtype, W):
    N, Hkv, D, B = 8, 2, 128, 4
    q, kn, vn, rk, rv, sp = ring_case(dtype, B, N, W, [100, 0, 7, 9], 4, Hkv, D, 1100, empty=0.25)
    path = [[0, 2, 3, 5, 6, 7, 0, 0], [1] + [0] * 7, [0] * 8, [8] + [0] * 7]
    n_path = [6, 1, 0, 1]
    pos = [[100, 500, 101, 102, 500, 103, 104, 105], [0] * 8, [7] * 8, [9] * 8]
    ring = [rk.cuda(), rv.cuda(), torch.from_numpy(sp).cuda()]
    cuda_lib.swa_tree_commit(kn.cuda(), vn.cuda(), i64(pos), i32(path), i32(n_path), *ring, W)
    assert cuda_lib.device_status() == cuda_lib.ERR_INVALID     # sequence 3 names node 8 of 8
    for b in range(3):
        for j in range(n_path[b]):
            node = path[b][j]
            p = pos[b][node]
            rk[b, p % W], rv[b, p % W], sp[b, p % W] = kn[b, node], vn[b, node], p
    assert torch.equal(ring[0].cpu(), rk) and torch.equal(ring[1].cpu(), rv) and np.array_equal(ring[2].cpu().numpy(), sp)
    # positions a ring cannot hold
    before = [t.clone() for t in ring]
    for p in (-1, 2 ** 31):
        cuda_lib.swa_tree_commit(kn[:1].cuda(), vn[:1].cuda(), i64([[0] * 7 + [p]]), i32([[0, 7] + [0] * 6]), i32([2]),
                                 ring[0][:1], ring[1][:1], ring[2][:1], W)
        assert cuda_lib.device_status() == cuda_lib.ERR_INVALID
    for a, b in zip(ring, before):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_drafting_step_by_step(cuda_lib, dtype):
    """Rotate, check a tree, commit a path, and go on: the committed state and the
    next outputs are those of the same tokens decoded one at a time."""
    B, N, Hq, Hkv, D, W, T0 = 2, 6, 8, 2, 64, 16, 40
    rot = cuda_lib.rope_config(32, theta=640000.0)
    n_tok = T0 + N
    # the tokens of the accepted path, by position, and other nodes beside them
    toks = [wl.normal((B, n_tok, h, D), 1200 + i, dtype).cuda() for i, h in enumerate((Hq, Hkv, Hkv))]
    tq, tk = cuda_lib.rope(toks[0], toks[1], rot)
    tv = toks[2]
    cap = n_tok + 1
    kc, vc = (torch.zeros(B * cap, Hkv, D, dtype=dtype, device="cuda") for _ in range(2))
    starts = i64([0, cap])
    for b in range(B):
        kc[b * cap:b * cap + T0], vc[b * cap:b * cap + T0] = tk[b, :T0], tv[b, :T0]
    ring = (torch.empty(B, W, Hkv, D, dtype=dtype, device="cuda"), torch.empty(B, W, Hkv, D, dtype=dtype, device="cuda"),
            torch.empty(B, W, dtype=torch.int32, device="cuda"))
    cuda_lib.swa_prefill(tq[:, :T0].contiguous(), tk[:, :T0].contiguous(), tv[:, :T0].contiguous(), W, ring=ring)
    seq_len = i32([T0, T0])
    one_ring, one_k, one_v = [t.clone() for t in ring], kc.clone(), vc.clone()
    # a tree: nodes 0, 2, 3, 5 are the path (depths 0..3), 1 and 4 alternatives
    depth, masks = [0, 0, 1, 2, 2, 3], [1, 2, 5, 13, 21, 45]
    on_path = [0, 2, 3, 5]
    draft = [wl.normal((B, N, h, D), 1300 + i, dtype).cuda() for i, h in enumerate((Hq, Hkv, Hkv))]
    for j, node in enumerate(on_path):
        for d, t in zip(draft, toks):
            d[:, node] = t[:, T0 + j]
    pos = i64([[T0 + d for d in depth]] * B)
    q, kn = cuda_lib.rope(draft[0], draft[1], rot, pos=pos)
    for j, node in enumerate(on_path):
        assert torch.equal(q[:, node], tq[:, T0 + j]) and torch.equal(kn[:, node], tk[:, T0 + j])
    vn = draft[2]
    mask = tr.mask_tensor([masks] * B, N).cuda()
    before = [t.clone() for t in (kc, vc, *ring)]
    oc, lc = cuda_lib.cross_decode_tree(q, kn, vn, kc, vc, starts, seq_len, T0, tree_mask=mask, want_lse=True)
    os_, ls = cuda_lib.swa_decode_tree(q, kn, vn, pos, *ring, W, tree_mask=mask, want_lse=True)
    for a, b in zip((kc, vc, *ring), before):
        assert torch.equal(a, b)
    path, n_path = i32([on_path + [0, 0]] * B), i32([4] * B)
    new_len = cuda_lib.cross_tree_commit(kn, vn, path, n_path, kc, vc, starts, seq_len)
    cuda_lib.swa_tree_commit(kn, vn, pos, path, n_path, *ring, W)
    # one at a time
    for j, node in enumerate(on_path):
        p = T0 + j
        for b in range(B):
            one_k[b * cap + p], one_v[b * cap + p] = tk[b, p], tv[b, p]
        qj = tq[:, p].contiguous()
        ocj, lcj = cuda_lib.cross_decode(qj, one_k, one_v, starts, i32([p + 1] * B), cap, want_lse=True)
        osj = cuda_lib.swa_decode(qj, tk[:, p].contiguous(), tv[:, p].contiguous(), i64([p] * B), *one_ring, W)
        # the two differ by the roundings of both: each within half a step of
        # its weights and its output (bf16), and 2^-12 of fp32 arithmetic
        tol = 2 * (2.0 ** -12 + (2 * tr.BF16_HALF if dtype == BF else 0)) * float(tv.abs().max())
        assert (oc[:, node].float() - ocj.float()).abs().max().item() <= tol
        assert (os_[:, node].float() - osj.float()).abs().max().item() <= tol
        assert (lc[:, :, node] - lcj).abs().max().item() <= 2.0 ** -11
    assert new_len.tolist() == [T0 + 4] * B
    for a, b in zip((kc, vc, *ring), (one_k, one_v, *one_ring)):
        assert torch.equal(a, b)
    # and on from there, with an outcome checked in 64 bits
    nxt = wl.normal((B, 1, Hq, D), 1400, dtype).cuda()
    o, lse = cuda_lib.cross_decode_tree(nxt, kn[:, 1:2].contiguous(), vn[:, 1:2].contiguous(), kc, vc, starts, new_len,
                                        cap, want_lse=True)
    ref = tr.cross_tree(nxt.cpu(), kn[:, 1:2].cpu(), vn[:, 1:2].cpu(), kc.cpu(), vc.cpu(), [0, cap], [T0 + 4] * B)
    tr.assert_tree(o, lse, ref, dtype)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("most", [512, 1 << 20])     # with clusters (bf16), with a workspace
def test_graph_replay_and_two_streams(cuda_lib, dtype, most):
    """Captured once, replayed on new inputs; and two calls at once on two streams,
    each with its own workspace."""
    lens, N, Hq, Hkv, D = [500, 64, 0], 9, 8, 2, 128
    cases = [cross_case(dtype, lens, N, Hq, Hkv, D, s, fill=0.0) for s in (1500, 1600)]
    starts = cases[0][5]
    rng = np.random.default_rng(5)
    masks = [[tr.random_tree(rng, N)[0] for _ in lens] for _ in cases]
    refs = [tr.cross_tree(*c[:5], starts, lens, m) for c, m in zip(cases, masks)]
    dev = [[t.cuda() for t in c[:5]] + [tr.mask_tensor(m, N).cuda()] for c, m in zip(cases, masks)]
    live = [t.clone() for t in dev[0]]
    ss, sl = i64(starts), i32(lens)
    n = cuda_lib.cross_decode_tree_workspace_size(len(lens), N, most, Hq, Hkv, D, dtype)
    assert (n == 0) == (dtype == BF and most == 512)

    def call(x, ws):
        return cuda_lib.cross_decode_tree(*x[:5], ss, sl, most, tree_mask=x[5], want_lse=True, workspace=ws)
    ws = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(live, ws[0])
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(live, ws[0])
    for i in (1, 0, 1):
        for a, b in zip(live, dev[i]):
            a.copy_(b)
        g.replay()
        tr.assert_tree(*out, refs[i], dtype, f"replay {i}")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i] = call(dev[i], ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        tr.assert_tree(*outs[i], refs[i], dtype, f"stream {i}")


@pytest.mark.parametrize("dtype", [BF, FP])
def test_node_positions_at_both_ends(cuda_lib, dtype):
    """A node near the largest position and one near the smallest do not see each other."""
    N, W = 4, 8
    q, kn, vn, rk, rv, sp = ring_case(dtype, 1, N, W, [5], 4, 2, 64, 780)
    pos = [[-2 ** 63, 2 ** 63 - 1, 3, -2 ** 63 + 1]]
    masks = [[15] * N]
    # in the plain form as positions apart: node 0 and 3 see 0 (and 3 itself), 1 and 2 themselves
    ref = tr.cross_tree(q[:, :2], kn[:, :2], vn[:, :2], kn[0, :0], vn[0, :0], [0], [0], [[1, 2]])
    o, lse = run_swa(cuda_lib, q, kn, vn, pos, rk, rv, sp, W, masks)
    tr.assert_tree(o[:, :2].contiguous(), lse[:, :, :2].contiguous(), ref, dtype)
    ref = tr.cross_tree(q, kn, vn, kn[0, :0], vn[0, :0], [0], [0], [[1, 2, 4, 9]])
    tr.assert_tree(o[:, 3:].contiguous(), lse[:, :, 3:].contiguous(), [x[:, 3:] if x.ndim == 4 else x[:, :, 3:] for x in ref], dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G", [(1, 1), (2, 4), (9, 1), (4, 4), (3, 8), (8, 4), (33, 1), (16, 4), (11, 8), (64, 2), (50, 4)])
def test_fp32_row_blocks(cuda_lib, N, G, D):
    """Every row block of the fp32 kernels, full and ragged: segments of many
    tiles, keys whose scores grow along the sequence (so maxima keep moving), and
    nodes that nobody sees, with NaN in K and V."""
    lens, Hkv = [2300, 900, 1, 64], 2
    q, kn, vn, kc, vc, starts = cross_case(FP, lens, N, Hkv * G, Hkv, D, 1500)
    for s, n in zip(starts, lens):
        kc[s:s + n] *= torch.linspace(0, 1, n)[:, None, None]
    rng = np.random.default_rng(N)
    masks = [tr.random_tree(rng, N)[0] for _ in lens]
    for i in range(N):
        masks[0][i] &= ~(1 << (N - 1))
    masks[1] = [0] * N
    kn[0, N - 1], vn[0, N - 1] = math.nan, math.nan
    ref = tr.cross_tree(q, torch.nan_to_num(kn), torch.nan_to_num(vn), kc, vc, starts, lens, masks)
    for most in (2300, 1 << 20):
        tr.assert_tree(*run_cross(cuda_lib, q, kn, vn, kc, vc, starts, lens, masks, max_len=most), ref, FP)
    B, W = 3, 200
    q, kn, vn, rk, rv, sp = ring_case(FP, B, N, W, [150, 1000, 0], Hkv * G, Hkv, D, 1600)
    pos = [[150 + i for i in range(N)], [1000 + 5 * i for i in range(N)], list(range(N))]
    ref = tr.swa_tree(q, kn, vn, pos, rk, rv, sp, W)
    tr.assert_tree(*run_swa(cuda_lib, q, kn, vn, pos, rk, rv, sp, W), ref, FP)


def test_offsets_beyond_32_bits(cuda_lib):
    """Rows whose element offset passes 2^32 in a cache of 4.4e9 elements."""
    Hq, Hkv, D, N = 16, 16, 128, 3
    rows = (1 << 21) + 100000
    kc, vc = (torch.zeros(rows, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
    starts, lens = [rows - 300, 5], [300, 200]
    for s, n, seed in zip(starts, lens, (1700, 1702)):
        kc[s:s + n], vc[s:s + n] = wl.normal((n, Hkv, D), seed).cuda(), wl.normal((n, Hkv, D), seed + 1).cuda()
    q, kn, vn = (wl.normal((2, N, Hq, D), 1710 + i) for i in range(3))
    o, lse = cuda_lib.cross_decode_tree(q.cuda(), kn.cuda(), vn.cuda(), kc, vc, i64(starts), i32(lens), 300, want_lse=True)
    parts = [torch.cat([c[s:s + n].cpu() for s, n in zip(starts, lens)]) for c in (kc, vc)]
    tr.assert_tree(o, lse, tr.cross_tree(q, kn, vn, *parts, [0, 300], lens), BF)
    path = i32([[2, 0, 1], [1, 0, 0]])
    at = i64([rows - 3, 205])
    new_len = cuda_lib.cross_tree_commit(kn.cuda(), vn.cuda(), path, i32([3, 1]), kc, vc, at, i32([0, 0]))
    assert new_len.tolist() == [3, 1]
    assert torch.equal(kc[-3:].cpu(), kn[0, [2, 0, 1]]) and torch.equal(vc[-3:].cpu(), vn[0, [2, 0, 1]])
    assert torch.equal(vc[205].cpu(), vn[1, 1])


def test_python_refusals(cuda_lib):
    q, kn, vn, kc, vc, starts = [t.cuda() if isinstance(t, torch.Tensor) else t
                                 for t in cross_case(BF, [8], 2, 4, 2, 64, 1800)]
    good = dict(q=q, k_nodes=kn, v_nodes=vn, k_cache=kc, v_cache=vc, seq_start=i64(starts), seq_len=i32([8]), max_len=8)
    cuda_lib.cross_decode_tree(**good)
    for name, bad in [("q", q.float()), ("q", q.cpu()), ("q", q.half()), ("q", q[0]), ("k_nodes", kn[:, :1]),
                      ("v_nodes", vn.transpose(2, 3).contiguous().transpose(2, 3)), ("k_cache", kc[:, :1]),
                      ("v_cache", vc[1:]), ("seq_start", i32(starts)), ("seq_len", i64([8])),
                      ("tree_mask", i32([[1, 3]])), ("n_nodes", i64([2])), ("n_nodes", i32([2, 2])), ("o", q[:, :1])]:
        with pytest.raises(ValueError):
            cuda_lib.cross_decode_tree(**{**good, name: bad})
    with pytest.raises(cuda_lib.YocoError):
        cuda_lib.cross_decode_tree(**{**good, "max_len": 1 << 20},
                                   workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        cuda_lib.cross_tree_commit(kn, vn, i64([[0, 1]]), i32([1]), kc, vc, i64(starts), i32([8]))
    sl = i32([8])
    with pytest.raises(cuda_lib.YocoError):
        cuda_lib.cross_tree_commit(kn, vn, i32([[0, 1]]), i32([1]), kc, vc, i64(starts), sl, new_len=sl)
