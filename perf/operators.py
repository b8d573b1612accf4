"""The drafted-token operators of the attention core and the rotary positions beside them, as a user calls them.

  rope               rotary positions of Q and K: half / interleaved pairs, part of the head, scaled frequencies; the gradient
  cross_decode_tree  attention of a tree of drafted tokens over the packed shared cache
  swa_decode_tree    the same over the self-decoder's sliding-window ring
  cross_tree_commit  the accepted path's K / V appended to the shared cache
  swa_tree_commit    the accepted path's K / V pushed into the ring

Shapes: 32 query / 8 KV heads of 128 over 64K-128K tokens and a window of 1024, the benchmark's; 4 / 2 heads of 64
and a window of 32, the tiny stack's; groups of 1 and 8 in the drawn cases.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    big = dict(dtype="bf16", Hq=32, Hkv=8, D=128)
    tiny = dict(dtype="fp32", Hq=4, Hkv=2, D=64)
    yarn = dict(theta=640000.0, scaling="by_parts", factor=16.0, orig_len=4096)
    return [
        # one decode step's new tokens of 16 sequences
        dict(name="rope_decode", op="rope", B=16, T=1, rot=128, layout="half", theta=640000.0, scaling="none",
             factor=1.0, orig_len=0, back=False, far=131072, **big),
        # a 32K prompt with frequencies stretched for long contexts
        dict(name="rope_prefill_32k", op="rope", B=1, T=32768, rot=128, layout="half", back=False, far=0, **yarn, **big),
        # training: the gradient of interleaved pairs over a quarter of the head, ragged length
        dict(name="rope_grad_part", op="rope", B=3, T=4099, rot=32, layout="interleaved", theta=10000.0, scaling="linear",
             factor=4.0, orig_len=0, back=True, far=0, **dict(big, dtype="fp32")),
        # the least a speculative decoder asks for: one drafted token over a short cache
        dict(name="cross_tree_1x2k", op="cross", B=1, N=1, lo=2047, hi=2047, chain=True, **big),
        # a served batch: 16 ragged contexts, up to 16 drafted tokens each
        dict(name="cross_tree_16x128k", op="cross", B=16, N=16, lo=65536, hi=131072, chain=False, **big),
        # one long context, a wide tree: tensor work and cache reads weigh alike
        dict(name="cross_tree_1x128k_64", op="cross", B=1, N=64, lo=131007, hi=131007, chain=False, **big),
        # one layer's window step of four sequences
        dict(name="swa_tree_4x16", op="swa", B=4, N=16, W=1024, filled=65536, chain=False, **big),
        # the largest window batch
        dict(name="swa_tree_64x48", op="swa", B=64, N=48, W=1024, filled=70000, chain=False, **big),
        # four accepted of 16 drafted, each of 16 sequences
        dict(name="cross_commit_16", op="cross_commit", B=16, N=16, lo=1024, hi=4096, **big),
        dict(name="cross_commit_256x64", op="cross_commit", B=256, N=64, lo=100, hi=700, **big),
        # the window layers' counterparts; the first in the tiny stack's shape
        dict(name="swa_commit_tiny", op="swa_commit", B=1, N=7, W=32, filled=272, **tiny),
        dict(name="swa_commit_64x48", op="swa_commit", B=64, N=48, W=1024, filled=70000, **big),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "cross", "cross", "cross", "swa", "swa", "cross_commit", "swa_commit"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    Hq, Hkv, D = rng.choice([(32, 8, 128), (32, 8, 128), (4, 2, 64), (8, 8, 64), (16, 2, 128), (4, 4, 128)])
    c = dict(op=op, dtype=dtype, Hq=Hq, Hkv=Hkv, D=D)
    if op == "rope":
        B = _log(rng, 1, 64)
        c.update(B=B, T=_log(rng, 1, max(1, 16384 // B)), rot=rng.choice([16, 32, 48, 64] + ([96, 128] if D == 128 else [])),
                 layout=rng.choice(["half", "interleaved"]), theta=rng.choice([10000.0, 640000.0, 5000000.0]),
                 scaling=rng.choice(["none", "linear", "ntk", "by_parts"]), factor=rng.choice([2.0, 8.0, 32.0]),
                 orig_len=rng.choice([2048, 4096]), back=rng.random() < 0.4, far=_log(rng, 1000, 1 << 20))
        return c
    if op == "cross":
        B, N = _log(rng, 1, 16), _log(rng, 1, 64)
        most = 131072 if dtype == "bf16" else 8192
        most = max(256, min(most, (1 << 20) // B, (1 << 24) // (B * N)))
        if dtype == "fp32":
            most = max(256, most // max(1, B * N // 16))
        hi = _log(rng, 200, most)
        c.update(B=B, N=N, lo=rng.randint(0, hi), hi=hi, chain=rng.random() < 0.3)
    elif op == "swa":
        W = rng.choice([32, 200, 1024, 1024])
        most = 64 if dtype == "bf16" else 8
        c.update(B=_log(rng, 1, most), N=_log(rng, 1, min(W, 64 if dtype == "bf16" else 24)), W=W,
                 filled=rng.choice([_log(rng, 1, W), _log(rng, W, 100000)]), chain=rng.random() < 0.3)
    elif op == "cross_commit":
        lo = _log(rng, 1, 2000)
        c.update(B=_log(rng, 1, 256), N=_log(rng, 1, 64), lo=lo, hi=lo + rng.randint(0, 300))
    else:
        W = rng.choice([64, 200, 1024])
        c.update(B=_log(rng, 1, 64), N=_log(rng, 1, 64), W=W, filled=_log(rng, 1, 100000))
    return c


def _shape_rng(case):
    """Lengths and node counts follow from the case alone, so that its work is known."""
    return random.Random("%s %s %s %s" % (case["op"], case["B"], case["N"], case.get("hi", case.get("filled"))))


def _ragged(case):
    """(context lengths, drafted tokens, accepted tokens) of each sequence."""
    r = _shape_rng(case)
    B, N = case["B"], case["N"]
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(B)] if "lo" in case else [case["filled"]] * B
    nodes = [N] + [r.randint(max(1, N // 2), N) for _ in range(B - 1)]
    taken = [r.randint(0 if B > 1 else 1, (n + 3) // 4) for n in nodes]
    return lens, nodes, taken


def _signed(x):
    return x - (1 << 64) if x >> 63 else x


def _trees(case, seed):
    """Random trees in parents-first order: each node's mask of visible nodes (its ancestors and itself) as 64 bits, and its depth."""
    r = random.Random(1000003 * seed + 17)
    _, nodes, _ = _ragged(case)
    N, masks, depths = case["N"], [], []
    for n in nodes:
        m, d = [0] * N, [0] * N
        for i in range(n):
            parent = i - 1 if case.get("chain") else r.randint(max(-1, i - 6), i - 1)
            m[i] = (m[parent] if parent >= 0 else 0) | 1 << i
            d[i] = d[parent] + 1 if parent >= 0 else 0
        masks.append([_signed(x) for x in m])
        depths.append(d)
    return masks, depths


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(7919 * seed + 11)
    dt, B, Hq, Hkv, D = DT[case["dtype"]], case["B"], case["Hq"], case["Hkv"], case["D"]

    def normal(*shape):
        t = torch.empty(shape, dtype=dt, device=dev)
        flat = t.view(-1)
        for i in range(0, flat.numel(), 1 << 28):
            part = flat[i:i + (1 << 28)]
            part.copy_(torch.randn(part.numel(), generator=g, device=dev, dtype=torch.float32))
        return t

    def ints(x, dtype):
        return torch.tensor(x, dtype=dtype, device=dev)

    s = {"case": case}
    if case["op"] == "rope":
        T = case["T"]
        s["q"], s["k"] = normal(B, T, Hq, D), normal(B, T, Hkv, D)
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device=dev, dtype=torch.int64)
        s["pos"] = start + torch.arange(T, device=dev)
        s["rot"] = None
        if own:
            import shared_kv_decoder_b200 as yoco
            s["rot"] = yoco.rope_config(case["rot"], theta=case["theta"], layout=case["layout"], scaling=case["scaling"],
                                        factor=case["factor"], orig_len=case["orig_len"])
        return s
    N = case["N"]
    lens, nodes, taken = _ragged(case)
    masks, depths = _trees(case, seed)
    s["k_nodes"], s["v_nodes"] = normal(B, N, Hkv, D), normal(B, N, Hkv, D)
    s["n_nodes"] = ints(nodes, torch.int32)
    if case["op"] in ("cross", "swa"):
        s["q"] = normal(B, N, Hq, D)
        s["mask"] = None if case["chain"] else ints(masks, torch.int64)
    else:
        r = random.Random(seed)
        s["path"] = ints([sorted(r.sample(range(n), t)) + [0] * (N - t) for n, t in zip(nodes, taken)], torch.int32)
        s["n_path"] = ints(taken, torch.int32)
    if "lo" in case:
        # every sequence owns room for its context and N more rows
        starts = [0]
        for x in lens:
            starts.append(starts[-1] + x + N)
        s["k_cache"], s["v_cache"] = normal(starts[-1], Hkv, D), normal(starts[-1], Hkv, D)
        s["seq_start"], s["seq_len"], s["max_len"] = ints(starts[:-1], torch.int64), ints(lens, torch.int32), max(lens)
        s["seq_cap"] = ints([x + N for x in lens], torch.int32)
    else:
        W, p0 = case["W"], case["filled"]
        s["ring_k"], s["ring_v"] = normal(B, W, Hkv, D), normal(B, W, Hkv, D)
        # slot s holds the newest position below p0 that is s modulo the window
        slot = torch.arange(W, device=dev)
        newest = p0 - 1 - (p0 - 1 - slot) % W
        s["slot_pos"] = torch.where(newest >= 0, newest, -1).to(torch.int32).repeat(B, 1).contiguous()
        s["node_pos"] = ints(depths, torch.int64) + p0
        if case["op"] == "swa_commit":  # positions along the path follow one another
            at = torch.arange(N, device=dev).expand(B, N)
            s["node_pos"].scatter_(1, s["path"].long(), p0 + torch.where(at < s["n_path"][:, None], at, 0))
    return s


def _inv_freq(case):
    """The frequencies in 64 bits, radians a position, and what cos and sin are multiplied by."""
    rot, f = case["rot"], case["factor"]
    theta = case["theta"]
    if case["scaling"] == "ntk":
        theta *= f ** (rot / (rot - 2))
    w = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        return w / f, 1.0
    if case["scaling"] == "by_parts":
        turns = case["orig_len"] * w / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return keep * w + (1 - keep) * w / f, 0.1 * math.log(f) + 1
    return w, 1.0


def _rotate(x, cos, sin, case):
    rot = case["rot"]
    y = x.float()
    r, rest = y[..., :rot], y[..., rot:]
    if case["layout"] == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, rest], -1).to(x.dtype)


def _plain_rope(s):
    case = s["case"]
    w, m = _inv_freq(case)
    angle = s["pos"][..., None].double() * w.cuda()
    cos, sin = (m * angle.cos()).float()[:, :, None], (m * angle.sin()).float()[:, :, None]
    if case["back"]:
        sin = -sin
    return _rotate(s["q"], cos, sin, case), _rotate(s["k"], cos, sin, case)


def _bits(mask, N):
    if mask is None:
        return torch.ones(N, N, dtype=torch.bool, device="cuda").tril()[None]
    return (mask[:, :, None] >> torch.arange(N, device="cuda")) & 1 != 0


def _attend(q, k, v, visible):
    """softmax(q k^T / sqrt(D)) v in 32 bits; rows that see nothing give 0 and a log-sum of -inf."""
    B, N, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    qf = q.float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    x = torch.matmul(qf, k.float().permute(0, 2, 3, 1)).view(B, Hkv, N, G, -1) / math.sqrt(D)
    x = x.masked_fill(~visible[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0, m)
    x = (x - m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, N * G, -1), v.float().transpose(1, 2)).view(B, Hkv, N, G, D)
    o = torch.where(l > 0, o / l, 0).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(q.dtype)
    return o, (l.log() + m).permute(0, 1, 3, 2, 4).reshape(B, Hq, N)


def _plain_cross(s):
    N = s["q"].shape[1]
    at = torch.arange(s["max_len"], device="cuda")
    rows = (s["seq_start"][:, None] + at).clamp(max=s["k_cache"].shape[0] - 1)
    live = torch.arange(N, device="cuda") < s["n_nodes"][:, None]
    context = (at < s["seq_len"][:, None])[:, None] & live[:, :, None]
    nodes = _bits(s["mask"], N) & live[:, None] & live[:, :, None]
    return _attend(s["q"], torch.cat([s["k_cache"][rows], s["k_nodes"]], 1),
                   torch.cat([s["v_cache"][rows], s["v_nodes"]], 1), torch.cat([context, nodes], -1))


def _plain_swa(s):
    N, W = s["q"].shape[1], s["case"]["W"]
    live = torch.arange(N, device="cuda") < s["n_nodes"][:, None]
    p, old = s["node_pos"][:, :, None], s["slot_pos"][:, None].long()
    ring = (old >= 0) & (old < p) & (old > p - W) & live[:, :, None]
    other = s["node_pos"][:, None]
    nodes = _bits(s["mask"], N) & live[:, None] & live[:, :, None] & (other <= p) & (other > p - W)
    return _attend(s["q"], torch.cat([s["ring_k"], s["k_nodes"]], 1), torch.cat([s["ring_v"], s["v_nodes"]], 1),
                   torch.cat([ring, nodes], -1))


def _accepted(s):
    B, N = s["path"].shape
    at = torch.arange(N, device="cuda").expand(B, N)
    take = at < s["n_path"][:, None]
    node = torch.arange(B, device="cuda")[:, None], s["path"].long()
    return at, take, node


def _plain_cross_commit(s):
    at, take, node = _accepted(s)
    rows = s["seq_start"][:, None] + s["seq_len"][:, None] + at
    for cache, nodes in ((s["k_cache"], s["k_nodes"]), (s["v_cache"], s["v_nodes"])):
        cache[rows] = torch.where(take[..., None, None], nodes[node], cache[rows])
    return s["k_cache"], s["v_cache"], s["seq_len"] + s["n_path"]


def _plain_swa_commit(s):
    at, take, node = _accepted(s)
    slots = node[0], (s["case"]["filled"] + at) % s["case"]["W"]
    for ring, nodes in ((s["ring_k"], s["k_nodes"]), (s["ring_v"], s["v_nodes"])):
        ring[slots] = torch.where(take[..., None, None], nodes[node], ring[slots])
    s["slot_pos"][slots] = torch.where(take, s["node_pos"][node].to(torch.int32), s["slot_pos"][slots])
    return s["ring_k"], s["ring_v"], s["slot_pos"]


def _own_run(s):
    import shared_kv_decoder_b200 as yoco
    op = s["case"]["op"]
    if op == "rope":
        return yoco.rope(s["q"], s["k"], s["rot"], pos=s["pos"], backward=s["case"]["back"])
    if op == "cross":
        return yoco.cross_decode_tree(s["q"], s["k_nodes"], s["v_nodes"], s["k_cache"], s["v_cache"], s["seq_start"],
                                      s["seq_len"], s["max_len"], tree_mask=s["mask"], n_nodes=s["n_nodes"], want_lse=True)
    if op == "swa":
        return yoco.swa_decode_tree(s["q"], s["k_nodes"], s["v_nodes"], s["node_pos"], s["ring_k"], s["ring_v"],
                                    s["slot_pos"], s["case"]["W"], tree_mask=s["mask"], n_nodes=s["n_nodes"], want_lse=True)
    if op == "cross_commit":
        new_len = yoco.cross_tree_commit(s["k_nodes"], s["v_nodes"], s["path"], s["n_path"], s["k_cache"], s["v_cache"],
                                         s["seq_start"], s["seq_len"], seq_cap=s["seq_cap"])
        return s["k_cache"], s["v_cache"], new_len
    yoco.swa_tree_commit(s["k_nodes"], s["v_nodes"], s["node_pos"], s["path"], s["n_path"], s["ring_k"], s["ring_v"],
                         s["slot_pos"], s["case"]["W"])
    return s["ring_k"], s["ring_v"], s["slot_pos"]


def run(state):
    if own:
        return _own_run(state)
    return {"rope": _plain_rope, "cross": _plain_cross, "swa": _plain_swa, "cross_commit": _plain_cross_commit,
            "swa_commit": _plain_swa_commit}[state["case"]["op"]](state)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rope":
        n = B * case["T"]
        return {"bytes": 2 * n * (Hq + Hkv) * D * size + 8 * n, "flops": 3 * n * (Hq + Hkv) * case["rot"]}
    lens, nodes, taken = _ragged(case)
    row, N = Hkv * D * size, case["N"]
    if case["op"].endswith("commit"):
        return {"bytes": sum(4 * t * row + 4 * t + 12 for t in taken), "flops": 0}
    if case["op"] == "swa":
        lens = [min(x, case["W"]) for x in lens]
    read = sum(2 * row * (x + n) + Hq * D * size * n + 8 * n for x, n in zip(lens, nodes))
    seen = sum(n * x + n * (n + 1) // 2 for x, n in zip(lens, nodes))
    return {"bytes": read + B * N * Hq * (D * size + 4), "flops": 4 * Hq * D * seen}


def _exact_attention(q, keys, values, see):
    """One sequence, head by head, in 64 bits: q [N, Hq, D], keys and values [L, Hkv, D], see [N, L] truth values."""
    N, Hq, D = q.shape
    o = torch.zeros(N, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((Hq, N), -math.inf, dtype=torch.float64, device="cuda")
    for g in range(keys.shape[1]):
        k, v = keys[:, g].double(), values[:, g].double()
        for h in range(g * (Hq // keys.shape[1]), (g + 1) * (Hq // keys.shape[1])):
            score = (q[:, h].double() @ k.T) * D ** -0.5
            score = torch.where(see, score, torch.full_like(score, -math.inf))
            lse[h] = torch.logsumexp(score, 1)
            weight = torch.where(see.any(1, keepdim=True), (score - lse[h][:, None]).exp(), torch.zeros_like(score))
            o[:, h] = weight @ v
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        rot, f = case["rot"], case["factor"]
        theta = case["theta"] * (f ** (rot / (rot - 2.0)) if case["scaling"] == "ntk" else 1.0)
        turn, size = [], 1.0
        for i in range(rot // 2):
            w = math.exp(-2.0 * i / rot * math.log(theta))
            if case["scaling"] == "linear":
                w /= f
            elif case["scaling"] == "by_parts":
                size = 1.0 + 0.1 * math.log(f)
                r = min(1.0, max(0.0, (case["orig_len"] * w / (2 * math.pi) - 1.0) / 31.0))
                w *= r + (1.0 - r) / f
            turn.append(-w if case["back"] else w)
        # a pair as one complex number, turned by its angle
        phase = torch.polar(torch.tensor(size, dtype=torch.float64, device="cuda"),
                            s["pos"].double()[..., None] * torch.tensor(turn, dtype=torch.float64, device="cuda"))[:, :, None]
        got = []
        for x in (s["q"], s["k"]):
            y = x.double()
            if case["layout"] == "half":
                z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * phase
                y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
            else:
                z = torch.complex(y[..., 0:rot:2].contiguous(), y[..., 1:rot:2].contiguous()) * phase
                y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
            got.append(y)
        return tuple(got)
    lens, nodes, taken = _ragged(case)
    B, N = case["B"], case["N"]
    if case["op"] in ("cross", "swa"):
        masks, depths = _trees(case, seed)
        os, ls = [], []
        for b in range(B):
            n = nodes[b]
            see = torch.zeros(N, lens[b] if case["op"] == "cross" else case["W"], dtype=torch.bool)
            if case["op"] == "cross":
                a = int(s["seq_start"][b])
                old_k, old_v = s["k_cache"][a:a + lens[b]], s["v_cache"][a:a + lens[b]]
                see[:n] = True
            else:
                old_k, old_v = s["ring_k"][b], s["ring_v"][b]
                held = s["slot_pos"][b].tolist()
                for i in range(n):
                    p = case["filled"] + depths[b][i]
                    see[i] = torch.tensor([0 <= old and 0 < p - old < case["W"] for old in held])
            tree = torch.zeros(N, N, dtype=torch.bool)
            for i in range(n):
                for j in range(n):
                    tree[i, j] = (masks[b][i] >> j) & 1 == 1
                    if case["op"] == "swa":
                        tree[i, j] &= 0 <= depths[b][i] - depths[b][j] < case["W"]
            o, l = _exact_attention(s["q"][b], torch.cat([old_k, s["k_nodes"][b]]), torch.cat([old_v, s["v_nodes"][b]]),
                                    torch.cat([see, tree], 1).cuda())
            os.append(o)
            ls.append(l)
        return torch.stack(os), torch.stack(ls)
    # the commits copy: what they write is exact in any type
    path = s["path"].tolist()
    if case["op"] == "cross_commit":
        for b in range(B):
            a = int(s["seq_start"][b]) + lens[b]
            for j in range(taken[b]):
                s["k_cache"][a + j] = s["k_nodes"][b, path[b][j]]
                s["v_cache"][a + j] = s["v_nodes"][b, path[b][j]]
        return s["k_cache"].double(), s["v_cache"].double(), torch.tensor([x + t for x, t in zip(lens, taken)], dtype=torch.int32)
    for b in range(B):
        for j in range(taken[b]):
            slot = (case["filled"] + j) % case["W"]
            s["ring_k"][b, slot] = s["k_nodes"][b, path[b][j]]
            s["ring_v"][b, slot] = s["v_nodes"][b, path[b][j]]
            s["slot_pos"][b, slot] = case["filled"] + j
    return s["ring_k"].double(), s["ring_v"].double(), s["slot_pos"]
