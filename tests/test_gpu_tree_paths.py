"""Tree attention on each way its kernels have of sharing the work -- clusters of
every size and the numbered shares, one row tile and two -- against plain 64-bit
forms."""
import numpy as np
import pytest
import torch

from tests import tree_ref as tr
from tests.test_gpu_tree import cross_case, run_cross

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
