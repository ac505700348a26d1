"""Operators around the caches of block-sparse decoding, as they are measured: rotary positions
(alone, into the caches with their gradient, and of draft trees), the verification of drafted
tokens, and the commit of the accepted ones.  `own` false: their plain form in elementary torch
operations; `own` true: the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

TWO_PI = 2.0 * math.pi


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of four sequences at 128K tokens: latency
        dict(name="rope_step_b4", op="rope", rows=4, Hq=32, Hkv=2, d=128, rot=128, inter=False, dtype="bf16",
             back=False, scaling="yarn", base=10000.0, far=131072),
        # the gradient of a 4096-token chunk's q and K, fp32 as the attention's backward gives it
        dict(name="rope_grad_4k", op="rope", rows=4096, Hq=32, Hkv=2, d=128, rot=128, inter=False, dtype="fp32",
             back=True, scaling="none", base=10000.0, far=32768),
        # ragged prompts of many sequences from one fused projection, part of the head, interleaved pairs
        dict(name="append_packed_8", op="append", B=8, tq=3001, L=16384, Hq=32, Hkv=2, d=128, rot=64, inter=True,
             packed=True, fused=True, scaling="ntk", base=10000.0),
        # whole prompts of 16K tokens
        dict(name="append_prompt_4x16k", op="append", B=4, tq=16384, L=16384, Hq=32, Hkv=2, d=128, rot=128, inter=False,
             packed=False, fused=False, scaling="none", base=10000.0),
        # gradients of a small odd batch, fp32 out
        dict(name="append_bwd_3x301", op="append_bwd", B=3, tq=301, L=2048, Hq=2, Hkv=1, d=64, rot=64, inter=False,
             packed=True, out="fp32", scaling="none", base=10000.0),
        # gradients of a 4096-token chunk over a 32K cache, bf16 out
        dict(name="append_bwd_4k", op="append_bwd", B=1, tq=4096, L=32768, Hq=32, Hkv=2, d=128, rot=128, inter=False,
             packed=False, out="bf16", scaling="yarn", base=10000.0),
        # one tree of 16 drafts after 64K tokens
        dict(name="drafts_16", op="drafts", B=1, n=16, L=65536, Hq=32, Hkv=2, d=128, rot=128, inter=False,
             scaling="yarn", base=10000.0),
        # four trees of 64 drafts, part of the head
        dict(name="drafts_4x64", op="drafts", B=4, n=64, L=65536, Hq=32, Hkv=2, d=128, rot=96, inter=True,
             scaling="none", base=1000000.0),
        # one tree of 16 drafts, siblings drawn without replacement, an odd vocabulary
        dict(name="verify_tree_16", op="verify", B=1, n=16, V=32001, branch=3, tree=True, dtype="fp32",
             drafts="distinct", sharp=2.5, near=0.7),
        # chains of a serving batch: seven drafts and their root each
        dict(name="verify_chain_64x8", op="verify", B=64, n=8, V=131072, branch=1, tree=False, dtype="fp32",
             drafts="replaced", sharp=3.0, near=0.5),
        # a handful of accepted tokens of one tree
        dict(name="commit_16", op="commit", B=1, n=16, L=65536, Hkv=2, d=128, bs=64, c=32, s=16),
        # a serving batch of deep chains, each completing kernels
        dict(name="commit_32x64", op="commit", B=32, n=64, L=4096, Hkv=8, d=128, bs=64, c=32, s=16),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "append_bwd", "drafts", "verify", "verify", "commit"])
    d = rng.choice([64, 128, 128])
    G, Hkv = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 8])
    heads = dict(Hq=G * Hkv, Hkv=Hkv, d=d)
    wheel = dict(rot=rng.choice([d, d, d // 2, d // 4, 3 * d // 4, 2 * rng.randint(1, d // 2)]),
                 inter=rng.random() < 0.5, scaling=rng.choice(["none", "none", "yarn", "ntk", "linear"]),
                 base=rng.choice([10000.0, 500000.0]))
    room = 65536 * 36 * 128  # elements of the largest listed case
    if op == "rope":
        most = max(2, min(16384, room // ((G + 1) * Hkv * d * 4)))
        return dict(op=op, rows=_between(rng, 1, most), dtype=rng.choice(["bf16", "fp32"]), back=rng.random() < 0.5,
                    far=_between(rng, 1024, 1 << 20), **heads, **wheel)
    if op in ("append", "append_bwd"):
        B = _between(rng, 1, 24)
        most = max(2, min(16384, room // (2 * (G + 2) * Hkv * d * B)))
        tq = _between(rng, 1, most)
        case = dict(op=op, B=B, tq=tq, L=tq + _between(rng, 1, 8192), packed=rng.random() < 0.6, **heads, **wheel)
        if op == "append":
            return dict(case, fused=rng.random() < 0.5)
        return dict(case, out=rng.choice(["bf16", "fp32"]))
    if op == "drafts":
        return dict(op=op, B=_between(rng, 1, 64), n=rng.randint(1, 64), L=_between(rng, 128, 1 << 20), **heads, **wheel)
    if op == "verify":
        tree = rng.random() < 0.6
        n = rng.randint(1, 64) if tree else rng.randint(1, 9)
        V = _between(rng, 100, 160000)
        B = _between(rng, 1, max(1.01, min(256, 64 * 8 * 131072 / (n * V * (3 if tree else 1)))))
        return dict(op=op, B=B, n=n, V=V, branch=rng.randint(1, 4) if tree else 1, tree=tree,
                    dtype=rng.choice(["fp32", "fp32", "bf16"]), drafts=rng.choice(["replaced", "distinct", "fixed"]),
                    sharp=rng.uniform(0.5, 5.0), near=rng.uniform(0.1, 1.5))
    c = rng.choice([16, 32, 32, 64, rng.randint(1, 64)])
    return dict(op=op, B=_between(rng, 1, 64), n=rng.randint(1, 64), L=_between(rng, 256, 8192), Hkv=Hkv, d=d, bs=64,
                c=c, s=rng.choice([16, max(1, c // 2), rng.randint(1, 64)]))


# ---------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "rope":
        e = case["rows"] * (case["Hq"] + case["Hkv"]) * case["d"]
        return dict(bytes=e * 2 * (2 if case["dtype"] == "bf16" else 4) + case["rows"] * 4, flops=3 * e)
    if op in ("append", "append_bwd"):
        e = _rows(case) * (case["Hq"] + 2 * case["Hkv"]) * case["d"]
        per = 4 if op == "append" else 4 + (2 if case["out"] == "bf16" else 4)
        return dict(bytes=e * per, flops=3 * e)
    if op == "drafts":
        e = case["B"] * case["n"] * (case["Hq"] + 2 * case["Hkv"]) * case["d"]
        return dict(bytes=e * 4, flops=3 * e)
    if op == "verify":
        # the last node's row of the target, and of the drafts where one of its children was rejected
        e = case["B"] * case["V"] * (1 if case["drafts"] == "fixed" or case["n"] == 1 else 2)
        return dict(bytes=e * (2 if case["dtype"] == "bf16" else 4), flops=2 * e)
    # about half of the drafts stand; the kernels they complete read c rows each
    rows = case["B"] * case["Hkv"] * (case["n"] + 1) / 2
    pooled = rows / case["s"]
    return dict(bytes=(rows * 4 + pooled * (case["c"] + 1)) * case["d"] * 2, flops=pooled * case["c"] * case["d"])


def _lengths(case):
    """Chunk lengths: all the same, or spread below the longest, one of them empty where there are several."""
    if not case["packed"]:
        return [case["tq"]] * case["B"]
    r = random.Random(case["tq"] * 1000 + case["B"])
    n = [r.randint(1, case["tq"]) for _ in range(case["B"])]
    n[0] = case["tq"]
    if case["B"] > 2:
        n[1] = 0
    return n


def _rows(case):
    return sum(_lengths(case))


# ---------------------------------------------------------------------------- inputs

def _theta(case):
    """Radians per position of each pair, in 64 bits, and the factor on the rotated elements."""
    rot, base = case["rot"], case["base"]
    i = np.arange(rot // 2, dtype=np.float64)
    scaling, factor = case["scaling"], 8.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    theta = base ** (-2.0 * i / rot)
    if scaling == "linear":
        theta = theta / factor
    if scaling == "yarn":
        at = [rot * math.log(4096 / (b * TWO_PI)) / (2 * math.log(base)) for b in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0, 1)
        return theta / factor * ramp + theta * (1 - ramp), 0.1 * math.log(factor) + 1
    return theta, 1.0


def _wheel(case):
    theta, scale = _theta(case)
    turns = np.floor(np.modf(theta / TWO_PI)[0] * 2.0 ** 64).astype(np.uint64)
    return dict(theta=torch.from_numpy(theta).cuda(), freqs=torch.from_numpy(turns.view(np.int64)).cuda(),
                rope=dict(rotary_dim=case["rot"], interleaved=int(case["inter"]), attn_scale=scale))


def _tree(r, n, branch, tree):
    """Parents of a draft tree whose node 0 is its root: a chain, or random with at most `branch` children."""
    parent, kids = [-1], [0] * n
    for i in range(1, n):
        free = [j for j in range(i) if kids[j] < branch]
        p = free[min(len(free) - 1, int(r.random() ** 2 * len(free)))] if tree else i - 1
        parent.append(p)
        kids[p] += 1
    return parent


def _masks(parents):
    rows = []
    for parent in parents:
        m = []
        for i, p in enumerate(parent):
            m.append((1 << i) | (m[p] if p >= 0 else 0))
        rows.append(m)
    return torch.from_numpy(np.array(rows, dtype=np.uint64).view(np.int64)).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)
    s = dict(case)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    op = case["op"]
    if op in ("rope", "append", "append_bwd", "drafts"):
        s |= _wheel(case)
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op == "rope":
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["q"], s["k"] = normal(case["rows"], Hq, d, dtype=t), normal(case["rows"], Hkv, d, dtype=t)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["pos"] = torch.randint(0, case["far"], (case["rows"],), generator=g, device="cuda", dtype=torch.int32)
    elif op in ("append", "append_bwd"):
        n = _lengths(case)
        total, B, L = sum(n), case["B"], case["L"]
        kv = [r.randint(max(x, 1), L) for x in n]
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda") if case["packed"] else None
        lead = (total,) if case["packed"] else (B, case["tq"])
        if op == "append":
            if case["fused"]:  # one projection's output, [q heads | k heads | v heads] in each row
                x = normal(*lead, Hq + 2 * Hkv, d)
                s["q"], s["k"], s["v"] = x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], x[..., Hq + Hkv:, :]
            else:
                s["q"], s["k"], s["v"] = normal(*lead, Hq, d), normal(*lead, Hkv, d), normal(*lead, Hkv, d)
            s["q_out"] = torch.empty((*lead, Hq, d), dtype=torch.bfloat16, device="cuda")
            s["k_cache"], s["v_cache"] = normal(B, Hkv, L, d), normal(B, Hkv, L, d)
        else:
            s["dq"] = normal(*lead, Hq, d, dtype=torch.float32)
            s["dk"], s["dv"] = normal(B, Hkv, L, d, dtype=torch.float32), normal(B, Hkv, L, d, dtype=torch.float32)
            t = torch.bfloat16 if case["out"] == "bf16" else torch.float32
            s["dq_out"] = torch.empty((*lead, Hq, d), dtype=t, device="cuda")
            s["dk_out"], s["dv_out"] = (torch.empty((*lead, Hkv, d), dtype=t, device="cuda") for _ in range(2))
    elif op == "drafts":
        B, n = case["B"], case["n"]
        s["tree_mask"] = _masks([_tree(r, n, 3, True) for _ in range(B)])
        s["kv_len"] = torch.tensor([r.randint(1, case["L"]) for _ in range(B)], dtype=torch.int32, device="cuda")
        x = normal(B, n, Hq + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], x[..., Hq + Hkv:, :]
        s["q_out"] = torch.empty((B, n, Hq, d), dtype=torch.bfloat16, device="cuda")
        s["draft_k"], s["draft_v"] = (torch.empty((B, Hkv, n, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    elif op == "verify":
        B, n, V = case["B"], case["n"], case["V"]
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        logits = torch.randn((B, n, V), generator=g, device="cuda") * case["sharp"]
        s["target"] = torch.softmax(logits, -1).to(t)
        logits += torch.randn((B, n, V), generator=g, device="cuda") * case["near"]
        draft = torch.softmax(logits, -1)
        del logits
        s["draft"] = None if case["drafts"] == "fixed" else draft.to(t)
        parents = [_tree(r, n, case["branch"], case["tree"]) for _ in range(B)]
        s["tree_mask"] = _masks(parents) if case["tree"] else None
        K = case["branch"]
        if case["drafts"] == "fixed":
            some = torch.topk(draft.view(B * n, V), K).indices.view(B, n, K)
        else:
            some = torch.multinomial(s["draft"].float().view(B * n, V), K, replacement=case["drafts"] == "replaced",
                                     generator=g).view(B, n, K)
        rank = [[p[:i].count(p[i]) for i in range(n)] for p in parents]
        at = torch.tensor([[max(x, 0) for x in p] for p in parents], device="cuda")
        rows = torch.arange(B, device="cuda")[:, None]
        s["tokens"] = some[rows, at, torch.tensor(rank, device="cuda")].to(torch.int32)
        s["u"] = torch.rand((B, n), generator=g, device="cuda")
        s["kv_len"] = torch.randint(1, 65536, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["path"], s["out_tokens"] = (torch.empty((B, n), dtype=torch.int32, device="cuda") for _ in range(2))
        s["n_path"], s["kv_len_out"] = (torch.empty((B,), dtype=torch.int32, device="cuda") for _ in range(2))
    else:
        B, n, L, Hkv, d = case["B"], case["n"], case["L"], case["Hkv"], case["d"]
        room = L + 2 * n
        s["draft_k"], s["draft_v"] = normal(B, Hkv, n, d), normal(B, Hkv, n, d)
        s["k_cache"], s["v_cache"] = normal(B, Hkv, room, d), normal(B, Hkv, room, d)
        M = (room + n - case["c"]) // case["s"] + 2
        s["kernel_cache"] = normal(B, Hkv, M, d)
        taken = [sorted(r.sample(range(n), r.randint(1, n))) for _ in range(B)]
        s["path"] = torch.tensor([x + [-1] * (n - len(x)) for x in taken], dtype=torch.int32, device="cuda")
        s["n_path"] = torch.tensor([len(x) for x in taken], dtype=torch.int32, device="cuda")
        s["kv_len"] = torch.tensor([r.randint(L // 2, L) + len(x) for x in taken], dtype=torch.int32, device="cuda")
        s["params"] = dict(block_size=case["bs"], kernel_size=case["c"], kernel_stride=case["s"], topk=8,
                           n_init_blocks=1, n_local_blocks=2, dense_len=0)
    return s


# ---------------------------------------------------------------------------- the operators

def run(state):
    if own:
        return _library(state)
    return _PLAIN[state["op"]](state)


def _library(s):
    from block_sparse_long_infllm_gb300 import infllmv2 as lib

    op = s["op"]
    if op == "rope":
        lib.rope(s["q"], s["k"], s["pos"], s["q_out"], s["k_out"], s["freqs"], s["rope"], transposed=s["back"])
        return s["q_out"], s["k_out"]
    if op == "append":
        lib.rope_append(s["q"], s["k"], s["v"], s["q_out"], s["k_cache"], s["v_cache"], s["kv_len"], s["freqs"],
                        s["rope"], cu_q=s["cu"], Tq_max=s["tq"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "append_bwd":
        lib.rope_append_bwd(s["dq"], s["dk"], s["dv"], s["dq_out"], s["dk_out"], s["dv_out"], s["kv_len"], s["freqs"],
                            s["rope"], cu_q=s["cu"], Tq_max=s["tq"])
        return s["dq_out"], s["dk_out"], s["dv_out"]
    if op == "drafts":
        lib.rope_drafts(s["q"], s["k"], s["v"], s["q_out"], s["draft_k"], s["draft_v"], s["kv_len"], s["tree_mask"],
                        s["freqs"], s["rope"])
        return s["q_out"], s["draft_k"], s["draft_v"]
    if op == "verify":
        lib.verify(s["tokens"], s["target"], s["draft"], s["u"], s["path"], s["n_path"], s["out_tokens"],
                   tree_mask=s["tree_mask"], kv_len=s["kv_len"], kv_len_out=s["kv_len_out"],
                   replace=s["drafts"] != "distinct")
        return s["path"], s["n_path"], s["out_tokens"], s["kv_len_out"]
    lib.commit(s["draft_k"], s["draft_v"], s["path"], s["n_path"], s["k_cache"], s["v_cache"], s["kernel_cache"],
               s["kv_len"], s["params"])
    return s["k_cache"], s["v_cache"], s["kernel_cache"]


def _turn(s, x, pos, back=False):
    """x [rows, heads, d] rotated at its rows' positions, in fp32 with the angles in 64 bits."""
    rot = s["rope"]["rotary_dim"]
    angle = pos.double()[:, None] * s["theta"]
    scale = s["rope"]["attn_scale"]
    cos, sin = (angle.cos() * scale).float()[:, None], (angle.sin() * scale).float()[:, None]
    if back:
        sin = -sin
    x = x.float()
    if s["rope"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_rope(s):
    return tuple(_turn(s, s[x], s["pos"], s["back"]).to(s[x].dtype) for x in ("q", "k"))


def _places(s):
    """Sequence and cache row of each token row."""
    kv = s["kv_len"].long()
    if s["cu"] is None:
        b = torch.arange(s["B"], device="cuda").repeat_interleave(s["tq"])
        return b, kv[b] - s["tq"] + torch.arange(s["tq"], device="cuda").repeat(s["B"])
    cu = s["cu"].long()
    rows = torch.arange(s["dq" if "dq" in s else "q"].shape[0], device="cuda")
    b = torch.searchsorted(cu, rows, right=True) - 1
    return b, kv[b] - cu[b + 1] + rows


def _plain_append(s):
    b, x = _places(s)
    q, k, v = (s[name].flatten(0, -3) for name in ("q", "k", "v"))
    s["q_out"].copy_(_turn(s, q, x).view_as(s["q_out"]))
    s["k_cache"][b, :, x] = _turn(s, k, x).bfloat16()
    s["v_cache"][b, :, x] = v
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_append_bwd(s):
    b, x = _places(s)
    t = s["dq_out"].dtype
    dq = _turn(s, s["dq"].flatten(0, -3), x, True).to(t)
    dk = _turn(s, s["dk"][b, :, x], x, True).to(t)
    dv = s["dv"][b, :, x].to(t)
    return dq.view_as(s["dq_out"]), dk.view_as(s["dk_out"]), dv.view_as(s["dv_out"])


def _bits(mask, n):
    """[B, n, n]: node i has node j on its way from the root, itself among them."""
    return ((mask[..., None] >> torch.arange(n, device="cuda")) & 1).bool()


def _plain_drafts(s):
    B, n = s["tree_mask"].shape
    x = (s["kv_len"].long()[:, None] + _bits(s["tree_mask"], n).sum(-1) - 1).flatten()
    q = _turn(s, s["q"].flatten(0, 1), x).bfloat16().view_as(s["q_out"])
    k = _turn(s, s["k"].flatten(0, 1), x).bfloat16().view(B, n, s["Hkv"], s["d"])
    return q, k.transpose(1, 2).contiguous(), s["v"].transpose(1, 2).contiguous()


def _plain_verify(s):
    """Every node tries its children in turn; the path is what hangs together from the root."""
    tokens, u, target = s["tokens"].long(), s["u"].double(), s["target"]
    B, n = tokens.shape
    node = torch.arange(n, device="cuda")
    if s["tree_mask"] is None:
        way = (node[:, None] >= node).expand(B, n, n)
    else:
        way = _bits(s["tree_mask"], n)
    parent = torch.where(way & (node != node[:, None]), node + 1, 0).amax(-1) - 1
    child = parent[:, None, :] == node[:, None]  # [b, node, child]
    rank = child.int().cumsum(-1) - 1
    at = parent.clamp(min=0)
    rows = torch.arange(B, device="cuda")[:, None]
    p = target[rows, at, tokens].double()
    fixed = s["draft"] is None
    q = torch.ones_like(p) if fixed else s["draft"][rows, at, tokens].double()
    c, Z, R = torch.zeros_like(p), torch.ones_like(p), torch.ones_like(p)
    taken = torch.full_like(tokens, -1)
    seen = torch.zeros((B, n, n), dtype=torch.bool, device="cuda")  # children rejected by each node
    same = tokens[:, :, None] == tokens[:, None, :]
    for k in range(s["branch"]):
        mine = child & (rank == k)
        has, ch = mine.any(-1) & (taken < 0), mine.int().argmax(-1)
        pk, qk, uk = p.gather(1, ch), q.gather(1, ch), u.gather(1, ch)
        if fixed:
            again = (seen & same.gather(1, ch[..., None].expand(B, n, n))).any(-1)
            w = torch.where(again, 0.0, pk)
        else:
            w = (pk - c * qk).clamp(min=0)
        stands = has & (uk * Z * qk < w * R)
        falls = has & ~stands
        taken = torch.where(stands, ch, taken)
        seen = seen | (mine & falls[..., None])
        if fixed:
            Z = torch.where(falls, (Z - w).clamp(min=0), Z)
            continue
        c = torch.where(falls & (R > 0), c + Z / R, c)
        if s["drafts"] == "distinct":
            R = torch.where(falls, R - qk, R)
        if k + 1 < s["branch"]:
            Z = torch.where(falls, (target.double() - c[..., None] * s["draft"].double()).clamp(min=0).sum(-1), Z)
    stood = (taken.gather(1, at) == node) | (node == 0)
    on = (stood[:, None, :] | ~way).all(-1)
    count = on.sum(-1)
    last = torch.where(on, node, 0).amax(-1)
    b = torch.arange(B, device="cuda")
    full = target[b, last].double()
    if fixed:
        gone = seen[b, last]  # its rejected children
        first = torch.where(gone, tokens, tokens.amax(-1, keepdim=True) * 0 + s["V"])
        w = torch.cat((full, full[:, :1]), 1).scatter(1, first, 0.0)[:, :s["V"]]
    else:
        w = (full - c[b, last][:, None] * s["draft"][b, last].double()).clamp(min=0)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, full)
    run_sum = w.cumsum(-1)
    final = (run_sum > u[:, :1] * run_sum[:, -1:]).int().argmax(-1)
    order = torch.where(on, node, n + node).sort(-1).values
    order = torch.where(order < n, order, -1)
    out = torch.full_like(tokens, -1)
    out[:, :-1] = torch.where(order[:, 1:] >= 0, tokens.gather(1, order[:, 1:].clamp(min=0)), -1)
    out[b, count - 1] = final
    return order.int(), count.int(), out.int(), s["kv_len"] + count.int()


def _plain_commit(s):
    kv, m = s["kv_len"].long(), s["n_path"].long()
    B, n = s["path"].shape
    b = torch.arange(B, device="cuda")[:, None]
    t = torch.minimum(torch.arange(n, device="cuda").expand(B, n), m[:, None] - 1)
    x, src = (kv - m)[:, None] + t, s["path"].long().gather(1, t)
    s["k_cache"][b, :, x] = s["draft_k"][b, :, src]
    s["v_cache"][b, :, x] = s["draft_v"][b, :, src]
    c, step = s["c"], s["s"]
    j0 = ((kv - m - c + step) // step).clamp(min=0)  # the first kernel that ends at or behind the first new row
    j = j0[:, None] + torch.arange((n - 1) // step + 1, device="cuda")
    done = j * step + c <= kv[:, None]
    tok = (j[..., None] * step + torch.arange(c, device="cuda")).clamp(max=s["k_cache"].shape[2] - 1)
    mean = s["k_cache"][b[..., None], :, tok].double().sum(2) / c  # [B, kernels, Hkv, d]
    j = j.clamp(max=s["kernel_cache"].shape[2] - 1)
    s["kernel_cache"][b, :, j] = torch.where(done[..., None, None], mean.bfloat16(), s["kernel_cache"][b, :, j])
    return s["k_cache"], s["v_cache"], s["kernel_cache"]


_PLAIN = dict(rope=_plain_rope, append=_plain_append, append_bwd=_plain_append_bwd, drafts=_plain_drafts,
              verify=_plain_verify, commit=_plain_commit)


# ---------------------------------------------------------------------------- in 64 bits, from the definitions

def _exact_turn(case, x, pos, sign=1.0):
    """Pairs as complex numbers times scale * exp(i * pos * theta)."""
    theta, scale = _theta(case)
    rot = case["rot"]
    x = x.double()
    wheel = torch.polar(torch.full((), scale, dtype=torch.float64, device="cuda"),
                        sign * torch.outer(pos.double(), torch.from_numpy(theta).cuda())).unsqueeze(1)
    y = x.clone()
    if case["inter"]:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * wheel
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * wheel
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        sign = -1.0 if case["back"] else 1.0
        return tuple(_exact_turn(case, s[x], s["pos"], sign) for x in ("q", "k"))
    if op in ("append", "append_bwd"):
        kv, outs, r = s["kv_len"].tolist(), [], 0
        q = (s["q"] if op == "append" else s["dq"]).flatten(0, -3)
        if op == "append":
            k, v, kc, vc = s["k"].flatten(0, -3), s["v"].flatten(0, -3), s["k_cache"].double(), s["v_cache"].double()
        for b, m in enumerate(_lengths(case)):
            x = torch.arange(kv[b] - m, kv[b], device="cuda")
            if op == "append":
                outs.append(_exact_turn(case, q[r:r + m], x))
                kc[b, :, kv[b] - m:kv[b]] = _exact_turn(case, k[r:r + m], x).transpose(0, 1)
                vc[b, :, kv[b] - m:kv[b]] = v[r:r + m].double().transpose(0, 1)
            else:
                outs.append((_exact_turn(case, q[r:r + m], x, -1.0),
                             _exact_turn(case, s["dk"][b, :, kv[b] - m:kv[b]].transpose(0, 1), x, -1.0),
                             s["dv"][b, :, kv[b] - m:kv[b]].transpose(0, 1).double()))
            r += m
        if op == "append":
            return torch.cat(outs).view_as(s["q_out"]), kc, vc
        return tuple(torch.cat([o[i] for o in outs]).view_as(s[x]) for i, x in enumerate(("dq_out", "dk_out", "dv_out")))
    if op == "drafts":
        depth = [[bin(m & (2 ** 64 - 1)).count("1") for m in row] for row in s["tree_mask"].tolist()]
        x = (torch.tensor(depth, device="cuda") - 1 + s["kv_len"][:, None]).flatten()
        turned = [_exact_turn(case, s[name].flatten(0, 1), x).view(*s[name].shape) for name in ("q", "k")]
        return turned[0], turned[1].transpose(1, 2), s["v"].double().transpose(1, 2)
    if op == "verify":
        return _exact_verify(case, s)
    kc, vc, kern = s["k_cache"].double(), s["v_cache"].double(), s["kernel_cache"].double()
    for b, (kv, m, path) in enumerate(zip(s["kv_len"].tolist(), s["n_path"].tolist(), s["path"].tolist())):
        for t in range(m):
            kc[b, :, kv - m + t] = s["draft_k"][b, :, path[t]].double()
            vc[b, :, kv - m + t] = s["draft_v"][b, :, path[t]].double()
        for end in range(kv - m + 1, kv + 1):  # a kernel is complete with the token that ends it
            if end >= case["c"] and (end - case["c"]) % case["s"] == 0:
                kern[b, :, (end - case["c"]) // case["s"]] = kc[b, :, end - case["c"]:end].mean(1)
    return kc, vc, kern


def _exact_verify(case, s):
    """One sequence after another, from the root down, with normalised distributions at each step."""
    B, n, V = case["B"], case["n"], case["V"]
    tokens, u, kv = s["tokens"].tolist(), s["u"].double().tolist(), s["kv_len"].tolist()
    paths, outs, counts = np.full((B, n), -1), np.full((B, n), -1), np.zeros(B, dtype=np.int64)
    masks = None if s["tree_mask"] is None else [[m & (2 ** 64 - 1) for m in row] for row in s["tree_mask"].tolist()]
    for b in range(B):
        kids = {}
        for i in range(1, n):
            up = i - 1 if masks is None else (masks[b][i] ^ (1 << i)).bit_length() - 1
            kids.setdefault(up, []).append(i)
        cur, path, emitted = 0, [0], []
        while True:
            p = s["target"][b, cur].double().cpu().numpy()
            q = None if s["draft"] is None else s["draft"][b, cur].double().cpu().numpy()
            whole, nxt = p, None
            norm = 1.0  # the target's rows are distributions up to their rounding
            for i in kids.get(cur, ()):
                x = tokens[b][i]
                if q is None:
                    if u[b][i] * norm < p[x]:
                        nxt = i
                        break
                    p = p.copy()
                    norm = max(norm - p[x], 0.0)
                    p[x] = 0.0
                    continue
                left = 1.0 if case["drafts"] == "replaced" else max(1.0 - gone, 0.0) if i != kids[cur][0] else 1.0
                if left > 0 and u[b][i] * norm * q[x] < p[x] * left:
                    nxt = i
                    break
                gone = q[x] + (gone if i != kids[cur][0] else 0.0)
                if left > 0:
                    p = np.maximum(p - q * (norm / left), 0.0)
                    norm = p.sum()
            if nxt is None:
                break
            cur = nxt
            path.append(cur)
            emitted.append(tokens[b][cur])
        if not p.sum() > 0:
            p = whole
        run_sum = np.cumsum(p)
        emitted.append(int(np.searchsorted(run_sum, u[b][0] * run_sum[-1], side="right")))
        paths[b, :len(path)], outs[b, :len(emitted)], counts[b] = path, emitted, len(path)
    to = lambda a: torch.from_numpy(np.asarray(a)).int()  # noqa: E731
    return to(paths), to(counts), to(outs), to(counts) + s["kv_len"].cpu()
