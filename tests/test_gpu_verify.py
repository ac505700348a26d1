"""Verification of draft trees on the GPU against the definition in exact rationals (whole outputs
have to be equal), the distribution it keeps, the commit of the accepted drafts, and the speculative
loop of rotary positions, tree decode, verification and commit as a serving program runs it, eager
and as a replayed CUDA graph."""
import numpy as np
import pytest

import oracle
from block_sparse_long_infllm_gb300 import synth

import spec_ref
from spec_ref import masks_of, random_tree

from harness import bf16_to_np_bits, lib, to_dev, torch_mod

pytestmark = pytest.mark.gpu

UNUSED = 12345


def _outputs(B, n):
    torch = torch_mod()
    full = lambda *s: torch.full(s, UNUSED, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(path=full(B, n), n_path=full(B), out_tokens=full(B, n))


def _probs(rng, rows, V, sharp):
    x = rng.standard_normal((rows, V)) * sharp
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def _masks_dev(parents, n):
    return to_dev(np.array([masks_of(p + [p_ for p_ in range(len(p) - 1, n - 1)]) for p in parents], dtype=np.uint64))


def _run(tokens, target, draft, u, **kw):
    B, n = tokens.shape
    out = _outputs(B, n)
    lib().verify(tokens, target, draft, u, out["path"], out["n_path"], out["out_tokens"], **kw)
    torch_mod().cuda.synchronize()
    return out


def _check(out, b, n, path, toks):
    assert out["n_path"][b].item() == len(path)
    assert out["path"][b].tolist() == path + [-1] * (n - len(path))
    assert out["out_tokens"][b].tolist() == toks + [-1] * (n - len(toks))


CASES = [  # B, n, V, branch, dtype, mode, sharp
    (1, 1, 1, 1, "fp32", "replaced", 1.0), (2, 2, 2, 1, "fp32", "replaced", 1.0), (3, 5, 3, 2, "bf16", "replaced", 0.5),
    (4, 9, 5, 4, "fp32", "distinct", 0.5), (4, 16, 31, 3, "fp32", "replaced", 1.0), (3, 64, 33, 4, "fp32", "distinct", 0.7),
    (3, 64, 100, 63, "fp32", "fixed", 0.5), (2, 33, 257, 3, "bf16", "distinct", 0.3), (2, 8, 1001, 2, "fp32", "fixed", 2.0),
    (1, 7, 2049, 3, "fp32", "distinct", 1.0), (1, 6, 4099, 3, "bf16", "replaced", 1.0), (2, 5, 9001, 4, "fp32", "replaced", 2.0),
    (1, 4, 20011, 3, "fp32", "distinct", 3.0)]


@pytest.mark.parametrize("B,n,V,branch,dtype,mode,sharp", CASES)
@pytest.mark.parametrize("seed", range(3))
def test_verify_matches_exact_rationals(cuda_lib, B, n, V, branch, dtype, mode, sharp, seed):
    torch = torch_mod()
    rng = np.random.default_rng(1000 * seed + n + V)
    t = torch.float32 if dtype == "fp32" else torch.bfloat16
    # few tries stand and many siblings are tried: the draft is far from the target
    target = torch.from_numpy(_probs(rng, B * n, V, sharp)).to(t)
    draft = torch.from_numpy(_probs(rng, B * n, V, sharp)).to(t)
    tp, dp = target.double().numpy().reshape(B, n, V), draft.double().numpy().reshape(B, n, V)
    nodes = rng.integers(1, n + 1, B).astype(np.int32) if seed else np.full(B, n, dtype=np.int32)
    parents = [random_tree(rng, int(m), branch) for m in nodes]
    tokens = rng.integers(0, V, (B, n)).astype(np.int32)
    for b in range(B):
        for i in range(1, nodes[b]):
            q = dp[b, parents[b][i]]
            if mode != "fixed":
                tokens[b, i] = rng.choice(V, p=q / q.sum())
            if mode == "distinct" and V > n:  # not again what a sibling drew
                sib = [tokens[b, j] for j in range(1, i) if parents[b][j] == parents[b][i]]
                while tokens[b, i] in sib:
                    tokens[b, i] = rng.integers(0, V)
    u = rng.random((B, n)).astype(np.float32)
    u[0, 0] = [0.0, np.float32(1 - 2 ** -24), 1.0][seed]
    kv = rng.integers(0, 1000, B).astype(np.int32)
    kv_dev = to_dev(kv)
    out = _run(to_dev(tokens), target.view(B, n, V).cuda(), None if mode == "fixed" else draft.view(B, n, V).cuda(),
               to_dev(u), tree_mask=_masks_dev(parents, n), n_nodes=to_dev(nodes), kv_len=kv_dev, kv_len_out=kv_dev,
               replace=mode != "distinct")
    assert lib().sync_status() == 0
    for b in range(B):
        m = int(nodes[b])
        path, toks = spec_ref.verify(tokens[b, :m].tolist(), parents[b], tp[b], None if mode == "fixed" else dp[b], u[b],
                                     mode != "distinct")
        _check(out, b, n, path, toks)
        assert kv_dev[b].item() == kv[b] + len(path)


def test_chain_without_masks_and_many_sequences(cuda_lib):
    """Chains need no masks; 300 sequences of an odd vocabulary, some idle."""
    rng = np.random.default_rng(8)
    B, n, V = 300, 4, 77
    target, near = _probs(rng, B * n, V, 1.0), _probs(rng, B * n, V, 1.0)
    draft = ((target + near) / 2).astype(np.float32)
    tokens = np.array([[rng.choice(V, p=d / d.sum()) for d in row] for row in draft.reshape(B, n, V).astype(np.float64)],
                      dtype=np.int32)
    tokens[:, 1:] = tokens[:, :-1].copy()  # token i + 1 was drawn from row i
    u = rng.random((B, n)).astype(np.float32)
    nodes = np.full(B, n, dtype=np.int32)
    nodes[::7] = 0
    out = _run(to_dev(tokens), to_dev(target).view(B, n, V), to_dev(draft).view(B, n, V), to_dev(u), n_nodes=to_dev(nodes))
    assert lib().sync_status() == 0
    seen = set()
    for b in range(B):
        if nodes[b] == 0:
            _check(out, b, n, [], [])
            continue
        path, toks = spec_ref.verify(tokens[b].tolist(), [-1, 0, 1, 2], target.reshape(B, n, V)[b],
                                     draft.reshape(B, n, V)[b], u[b], True)
        _check(out, b, n, path, toks)
        seen.add(len(path))
    assert seen == {1, 2, 3, 4}


@pytest.mark.parametrize("dtype,V", [("fp32", 33001), ("bf16", 33003), ("fp32", 16384)])
@pytest.mark.parametrize("mode", ["replaced", "distinct", "fixed"])
def test_every_batch_size_decides_alike(cuda_lib, dtype, V, mode):
    """A sequence's row is spread over 16 CTAs when it is alone, 8 among 20, 4 among 100, one among 700: sums
    are exact, so its outputs are the same; two of them against the exact rationals."""
    torch = torch_mod()
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    B, n = 6, 4
    t = torch.float32 if dtype == "fp32" else torch.bfloat16
    logits = torch.randn((B, n, V), generator=g, device="cuda") * 2.0
    target = torch.softmax(logits, -1).to(t)
    draft = torch.softmax(logits + torch.randn((B, n, V), generator=g, device="cuda"), -1)
    tokens = torch.zeros((B, n), dtype=torch.int32, device="cuda")
    tokens[:, 1:] = torch.multinomial(draft[:, 0], 3, replacement=mode == "replaced", generator=g).int()
    draft = draft.to(t)
    u = torch.rand((B, n), generator=g, device="cuda")
    u[0, 1:], u[1, 1:] = 0.9999, 0.9999  # all three siblings are tried
    parents = [-1, 0, 0, 0]
    masks = to_dev(np.array([masks_of(parents)] * B, dtype=np.uint64))
    outs = []
    for copies in (1, 20, 100, 700):
        for b in range(B):
            rep = lambda x: x[b:b + 1].expand(copies, *x.shape[1:]).clone(memory_format=torch.contiguous_format)  # noqa: E731
            out = _run(rep(tokens), rep(target), None if mode == "fixed" else rep(draft), rep(u), tree_mask=rep(masks),
                       replace=mode != "distinct")
            assert all(torch.equal(out[k], out[k][:1].expand_as(out[k])) for k in out)
            outs.append({k: x[0].tolist() for k, x in out.items()})
    assert lib().sync_status() == 0
    for i in range(B, len(outs)):
        assert outs[i] == outs[i % B]
    for b in range(2):
        path, toks = spec_ref.verify(tokens[b].tolist(), parents, target[b].double().cpu().numpy(),
                                     None if mode == "fixed" else draft[b].double().cpu().numpy(), u[b].cpu().numpy(),
                                     mode != "distinct")
        assert outs[b]["path"][:len(path)] == path and outs[b]["out_tokens"][:len(toks)] == toks
        assert outs[b]["n_path"] == len(path)


def _one(target, draft, tokens, u, parents, **kw):
    """One sequence given as lists of rows."""
    n = len(tokens)
    f = lambda x: to_dev(np.array(x, dtype=np.float32))[None]  # noqa: E731
    out = _run(to_dev(np.array([tokens], dtype=np.int32)), f(target), None if draft is None else f(draft), f(u),
               tree_mask=_masks_dev([parents], n), **kw)
    k = out["n_path"].item()
    return out["path"][0, :k].tolist(), out["out_tokens"][0, :k].tolist()


def test_verify_at_its_borders(cuda_lib):
    half, a = [0.5, 0.5, 0, 0], [0.25, 0.25, 0.25, 0.25]
    # equal rows: every draft stands, even for u next to 1; dyadic borders: a token takes [lower, upper)
    assert _one([half] * 3, [half] * 3, [0, 1, 0], [0.5, 1 - 2 ** -24, 1 - 2 ** -24], [-1, 0, 1]) == ([0, 1, 2], [1, 0, 1])
    assert _one([a], [a], [0], [0.25], [-1]) == ([0], [1])
    assert _one([a], [a], [0], [np.nextafter(np.float32(0.25), np.float32(0))], [-1]) == ([0], [0])
    assert _one([[0, 0, 1, 0]], None, [0], [0.0], [-1]) == ([0], [2])   # weight 0 is never drawn
    assert _one([[0, 1, 0, 0]], None, [0], [1.0], [-1]) == ([0], [1])   # nor past the last weight
    # u = 0 stands wherever p > 0; p = 0 never stands; q = 0 at a drafted token stands wherever p > 0
    assert _one([half] * 2, [a] * 2, [0, 1], [0.0, 0.0], [-1, 0]) == ([0, 1], [1, 0])
    assert _one([half] * 2, [a] * 2, [0, 3], [0.0, 0.0], [-1, 0]) == ([0], [0])
    assert _one([half] * 2, [[0, 0, 1, 0]] * 2, [0, 1], [0.0, 0.9], [-1, 0]) == ([0, 1], [1, 0])
    # u q = p exactly is a rejection; the rest is p - q
    assert _one([[0.25, 0.75, 0, 0]] * 2, [[0.5, 0.5, 0, 0]] * 2, [0, 0], [0.0, 0.5], [-1, 0]) == ([0], [1])
    # nothing left after the rejection (q covers p): the draw is from p
    assert _one([[0.5, 0.25, 0, 0]] * 2, [[0.5, 0.25, 0.25, 0]] * 2, [0, 2], [0.9, 0.0], [-1, 0]) == ([0], [1])
    # without replacement, a first draft that held all of q leaves nothing for its siblings
    q1 = [0, 0, 1, 0]
    assert _one([half] * 3, [q1] * 3, [0, 2, 0], [0.7, 0.0, 0.0], [-1, 0, 0], replace=False) == ([0], [1])
    # chosen drafts: a rejected token is out for good, its twin too
    assert _one([half] * 3, None, [0, 0, 0], [0.0, 0.6, 0.0], [-1, 0, 0]) == ([0], [1])
    assert _one([half] * 3, None, [0, 0, 1], [0.0, 0.6, 0.999], [-1, 0, 0]) == ([0, 2], [1, 0])
    assert lib().sync_status() == 0


def test_weights_that_cancel_after_a_quotient_leave_nothing(cuda_lib):
    """Without replacement, with twins among the siblings: one token has all of w, and the drafts have nothing
    but it left, so the next rejection takes all of it, to the last unit although Z/R is no binary
    fraction.  The last token then comes from p."""
    # Z = 0.2578125, R = q(1) = 0.47265625
    p, q = [0.267578125, 0.73046875], [0.52734375, 0.47265625]
    tokens, parents, u = [0] * 5, [-1, 0, 0, 0, 0], [0.0341401, 0.9172202, 0.9963093, 0.9445311, 0.9634557]
    want = spec_ref.verify(tokens, parents, [p] * 5, [q] * 5, u, False)
    assert want == ([0], [0])
    assert _one([p] * 5, [q] * 5, tokens, u, parents, replace=False) == want
    # rows of 2 to 4 tokens in 512ths; siblings take the tokens in turn, then again from the first
    rng = np.random.default_rng(29)
    for V in (2, 3, 4):
        B, n = 400, 2 * V + 1
        cuts = np.sort(rng.integers(0, 513, (2, B, V - 1)), -1)
        rows = np.diff(np.concatenate([np.zeros((2, B, 1)), cuts, np.full((2, B, 1), 512)], -1), axis=-1) / 512
        target, draft = (np.repeat(r[:, None], n, 1).astype(np.float32) for r in rows)
        tokens = np.zeros((B, n), dtype=np.int32)
        for b in range(B):
            order = rng.permutation(V)
            tokens[b, 1:] = np.concatenate([order[:V - 1], order[:V - 1], order[:2]])
        u = (1 - rng.random((B, n)) * 1e-3).astype(np.float32)
        u[:, 0] = rng.random(B)
        masks = to_dev(np.array([masks_of([-1] + [0] * (n - 1))] * B, dtype=np.uint64))
        out = _run(to_dev(tokens), to_dev(target), to_dev(draft), to_dev(u), tree_mask=masks, replace=False)
        for b in range(B):
            _check(out, b, n, *spec_ref.verify(tokens[b].tolist(), [-1] + [0] * (n - 1), target[b].astype(np.float64),
                                               draft[b].astype(np.float64), u[b], False))
    assert lib().sync_status() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_of_few_tokens_at_the_tensors_end(cuda_lib, dtype):
    """Vocabularies of 1 to 17: several rows share the last 16 bytes of the tensor, and the path ends at
    each of them in turn."""
    torch = torch_mod()
    t = torch.float32 if dtype == "fp32" else torch.bfloat16
    for V in range(1, 18):
        rng = np.random.default_rng(V)
        n = 9
        target = torch.from_numpy(_probs(rng, n, V, 0.5)).to(t)
        draft = torch.from_numpy(_probs(rng, n, V, 0.5)).to(t)
        tp, dp = target.double().numpy(), draft.double().numpy()
        parents = [-1] + list(range(n - 1))
        tokens = rng.integers(0, V, (n, n)).astype(np.int32)
        u = np.zeros((n, n), dtype=np.float32)  # every draft stands ...
        u[:, 0] = rng.random(n)
        for b in range(n - 1):
            u[b, b + 1] = 1.0                   # ... up to node b
        rows = lambda x: x.expand(n, n, V).contiguous().cuda()  # noqa: E731
        out = _run(to_dev(tokens), rows(target), rows(draft), to_dev(u))
        for b in range(n):
            _check(out, b, n, *spec_ref.verify(tokens[b].tolist(), parents, tp, dp, u[b], True))
    assert lib().sync_status() == 0


def test_rejected_siblings_past_the_drafts_weight_change_nothing(cuda_lib):
    """Without replacement R stays at nothing once the rejected siblings' q have used it up, however far
    their sum goes past it: duplicates of a drafted token (sums from 2 to 62), and rows above 1."""
    one, other = [1.0, 0.0, 0.0, 0.0], [0.0, 1.0, 0.0, 0.0]
    for twins in range(2, 63):
        n = twins + 2
        tokens, parents, u = [0] * (n - 1) + [1], [-1] + [0] * (n - 1), [0.5] * n
        want = spec_ref.verify(tokens, parents, [other] * n, [one] * n, u, False)
        assert want == ([0], [1])
        assert _one([other] * n, [one] * n, tokens, u, parents, replace=False) == want
    big, p = [7.0, 0.75, 0.75, 0.0], [0.0, 0.25, 0.25, 0.5]  # 7 is read as 1
    tokens, parents, u = [0, 0, 1, 2, 0, 3, 3], [-1] + [0] * 6, [0.5, 0.5, 0.9, 0.9, 0.5, 0.0, 0.5]
    want = spec_ref.verify(tokens, parents, [p] * 7, [big] * 7, u, False)
    assert want == ([0], [3])
    assert _one([p] * 7, [big] * 7, tokens, u, parents, replace=False) == want
    assert lib().sync_status() == 0


def test_verify_reads_bad_numbers_as_documented(cuda_lib):
    nan, inf = float("nan"), float("inf")
    assert _one([[nan, 0.5, -1.0, 0.5]], None, [0], [0.0], [-1]) == ([0], [1])
    assert _one([[nan, -inf, 0.25, 0.75]], None, [0], [0.3], [-1]) == ([0], [3])
    assert _one([[0.0, inf, 0.0, 0.0]], None, [0], [0.5], [-1]) == ([0], [1])        # inf is read as 1
    assert _one([[0.0, 0.5, 0.5, 0.0]], None, [0], [nan], [-1]) == ([0], [1])        # u NaN is read as 0
    # rows that no step visits may hold anything
    half, junk = [0.5, 0.5, 0, 0], [nan] * 4
    # (node 1's token has p = q = 0: rejected, then w = p - q = 0 everywhere and node 2 falls too)
    assert _one([half, junk, half], [half, junk, junk], [0, 3, 1], [0.6, 0.0, 0.0], [-1, 0, 0]) == ([0], [1])
    # (p = 0 at node 1's token; w = (0.5, 0, 0, 0) is left and q = 0 at node 2's token, which stands)
    q = [0, 0.5, 0.25, 0.25]
    assert _one([half, junk, half], [q, junk, junk], [0, 3, 0], [0.6, 0.0, 0.9], [-1, 0, 0]) == ([0, 2], [0, 1])
    assert lib().sync_status() == 0


@pytest.mark.parametrize("replace", [True, False])
def test_draft_rows_of_bad_numbers_are_read_as_documented(cuda_lib, replace):
    """NaN, infinite, negative and large values in the draft rows of visited nodes (and NaN and negative ones in
    the target's), against the exact rationals, which read them as the header says."""
    nan, inf = float("nan"), float("inf")
    bad = [nan, inf, -inf, -0.5, 7.0, 1e38, -0.0, 1e-40]
    # by hand: q(1) = inf is read as 1 and p - q leaves token 0; q(1) = NaN or below 0 is 0 and token 1 stands
    half = [0.5, 0.5, 0.0, 0.0]
    for q, want in ((inf, ([0], [0])), (7.0, ([0], [0])), (nan, ([0, 1], [1, 0])), (-1.0, ([0, 1], [1, 0]))):
        assert _one([half] * 2, [[0.25, q, 0, 0]] * 2, [0, 1], [0.0, 0.75], [-1, 0], replace=replace) == want
    rng = np.random.default_rng(17)
    lengths = set()
    for _ in range(60):
        n, V = 8, 6
        target, draft = _probs(rng, n, V, 1.0), _probs(rng, n, V, 1.0)
        for row in range(n):
            draft[row, rng.choice(V, 2, replace=False)] = rng.choice(bad, 2)
            target[row, rng.integers(V)] = rng.choice([nan, -inf, -1.0, 0.25])
        parents = random_tree(rng, n, 4)
        tokens = rng.integers(0, V, n).tolist()
        u = rng.random(n).astype(np.float32).tolist()
        want = spec_ref.verify(tokens, parents, target, draft, u, replace)
        assert _one(target, draft, tokens, u, parents, replace=replace) == want
        lengths.add(len(want[0]))
    assert len(lengths) > 1
    assert lib().sync_status() == 0


def test_verify_reports_bad_sequences_and_keeps_the_others(cuda_lib):
    torch = torch_mod()
    L = lib()
    B, n, V = 9, 3, 40
    target = torch.full((B, n, V), 1.0 / V, device="cuda")
    draft = target.clone()
    tokens = torch.ones((B, n), dtype=torch.int32, device="cuda")
    u = torch.zeros((B, n), device="cuda")
    masks = np.array([[1, 3, 7]] * B, dtype=np.uint64)
    masks[1, 0] = 3            # a root with a parent
    masks[2, 1] = 1            # without its own bit
    masks[3, 2] = 6            # not below the root
    masks[4, 1] = 7            # a parent behind its child
    tokens[5, 2] = V
    tokens[6, 1] = -1
    nodes = torch.full((B,), n, dtype=torch.int32, device="cuda")
    nodes[7] = n + 1
    target[8] = 0.1            # sums to 4
    kv = torch.arange(10, 10 + B, dtype=torch.int32, device="cuda")
    kv_out = torch.zeros_like(kv)
    out = _run(tokens, target, draft, u, tree_mask=to_dev(masks), n_nodes=nodes, kv_len=kv, kv_len_out=kv_out)
    assert L.sync_status() == L.ERR_DEVICE_INDEX
    _check(out, 0, n, [0, 1, 2], [1, 1, 0])
    assert kv_out.tolist() == [13] + list(range(11, 10 + B))
    for b in range(1, B):
        _check(out, b, n, [], [])
    target[8] = 0.0            # and a row of nothing
    out = _run(tokens[8:], target[8:].clone(), draft[8:].clone(), u[8:], tree_mask=to_dev(masks[8:]))
    assert L.sync_status() == L.ERR_DEVICE_INDEX
    _check(out, 0, n, [], [])
    assert L.sync_status() == 0


@pytest.mark.parametrize("mode", ["replaced", "distinct", "fixed"])
def test_verify_keeps_the_targets_distribution(cuda_lib, mode):
    """The first new token is distributed as the target's first row, whatever the drafts: 200,000
    sequences with three siblings each; every frequency within 5 standard deviations."""
    torch = torch_mod()
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    B, n, V = 200000, 4, 12
    p = torch.softmax(torch.randn(V, generator=g, device="cuda"), -1)
    q = torch.softmax(torch.randn(V, generator=g, device="cuda"), -1)
    tokens = torch.zeros((B, n), dtype=torch.int32, device="cuda")
    if mode == "fixed":
        tokens[:, 1:] = torch.topk(q, 3).indices.int()
    else:
        tokens[:, 1:] = torch.multinomial(q.expand(B, V), 3, replacement=mode == "replaced", generator=g).int()
    target, draft = p.expand(B, n, V).contiguous(), q.expand(B, n, V).contiguous()
    u = torch.rand((B, n), generator=g, device="cuda")
    masks = to_dev(np.array([1, 3, 5, 9], dtype=np.uint64)).expand(B, n).contiguous()
    out = _run(tokens, target, None if mode == "fixed" else draft, u, tree_mask=masks, replace=mode != "distinct")
    assert lib().sync_status() == 0
    freq = torch.bincount(out["out_tokens"][:, 0].long(), minlength=V).double() / B
    pd = p.double()
    assert bool(((freq - pd).abs() <= 5 * (pd * (1 - pd) / B).sqrt()).all())
    assert 0.2 < float((out["n_path"] == 2).double().mean()) < 1.0


def test_verify_past_32_bits(cuda_lib):
    """Probabilities of more than 2^32 elements: 65 chains of 64 over 2^20 tokens, each 2^-20."""
    torch = torch_mod()
    B, n, V = 65, 64, 1 << 20
    target = torch.full((B, n, V), 2.0 ** -20, dtype=torch.bfloat16, device="cuda")
    tokens = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n) * 200 % V
    u = torch.zeros((B, n), device="cuda")        # every draft stands
    u[:, 0] = torch.arange(B, device="cuda") / B  # and the last token is V b / B
    u[B - 1, n - 1] = 2.0 ** -20                   # but the last sequence's last: u = p is a rejection
    out = _run(tokens, target, None, u)
    assert lib().sync_status() == 0
    last = (u[:, 0].double() * V).long()
    for b in (0, 1, 37, B - 2):
        _check(out, b, n, list(range(n)), tokens[b, 1:].tolist() + [last[b].item()])
    # the rejected token weighs nothing: of the other V - 1, equally likely, that of u
    at = int(u[B - 1, 0].double().item() * (V - 1))
    at += at >= tokens[B - 1, n - 1].item()
    _check(out, B - 1, n, list(range(n - 1)), tokens[B - 1, 1:n - 1].tolist() + [at])


def test_verify_on_a_captured_graph_and_another_stream(cuda_lib):
    """Two captured graphs on two streams at once, replayed with new numbers, against eager calls."""
    torch = torch_mod()
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    sets = []
    for i in range(2):
        B, n, V = 3 + i, 6, 30011
        target = torch.softmax(torch.randn((B, n, V), generator=g, device="cuda"), -1)
        draft = torch.softmax(torch.randn((B, n, V), generator=g, device="cuda"), -1)
        tokens = torch.randint(0, V, (B, n), generator=g, device="cuda", dtype=torch.int32)
        s = dict(tokens=tokens, target=target, draft=draft, u=torch.rand((B, n), generator=g, device="cuda"),
                 out=_outputs(B, n), stream=torch.cuda.Stream(), graph=torch.cuda.CUDAGraph())
        call = lambda s=s: lib().verify(s["tokens"], s["target"], s["draft"], s["u"], *s["out"].values())  # noqa: E731
        torch.cuda.synchronize()
        with torch.cuda.stream(s["stream"]):
            call()
        torch.cuda.synchronize()
        with torch.cuda.graph(s["graph"], stream=s["stream"]):
            call()
        sets.append(s)
    for _ in range(5):
        for s in sets:
            s["u"].copy_(torch.rand(s["u"].shape, generator=g, device="cuda"))
        torch.cuda.synchronize()
        for s in sets:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
        torch.cuda.synchronize()
        for s in sets:
            eager = _run(s["tokens"], s["target"], s["draft"], s["u"])
            assert all(torch.equal(eager[k], s["out"][k]) for k in eager)
    assert lib().sync_status() == 0


# ---- commit

@pytest.mark.parametrize("B,n,Hkv,d,c,s,L", [(1, 1, 1, 64, 32, 16, 70), (2, 5, 2, 128, 32, 16, 300), (3, 64, 2, 64, 64, 1, 200),
                                             (4, 16, 3, 128, 17, 5, 150), (2, 64, 1, 128, 1, 1, 130), (2, 33, 2, 64, 33, 64, 260)])
def test_commit_matches_definition(cuda_lib, B, n, Hkv, d, c, s, L):
    torch = torch_mod()
    rng = np.random.default_rng(n + d)
    p = dict(block_size=64, kernel_size=c, kernel_stride=s, topk=4, n_init_blocks=1, n_local_blocks=2, dense_len=0)
    bits = lambda *sh: synth.f32_to_bf16_bits(rng.standard_normal(sh).astype(np.float32))  # noqa: E731
    k0, v0, dk, dv = bits(B, Hkv, L, d), bits(B, Hkv, L, d), bits(B, Hkv, n, d), bits(B, Hkv, n, d)
    M = max((L - c) // s + 1, 1)
    kern0 = bits(B, Hkv, M, d)
    for step in range(6):
        m = rng.integers(0, n + 1, B).astype(np.int32)
        if step == 0:
            m[0] = n
        kv = np.array([int(rng.integers(x, L + 1)) for x in m], dtype=np.int32)
        if step == 1:
            kv[0] = m[0]  # a sequence that starts empty
        if step == 2:
            kv[0] = L     # one that fills the cache
        path = np.full((B, n), -1, dtype=np.int32)
        for b in range(B):
            path[b, :m[b]] = np.sort(rng.choice(n, m[b], replace=False))
        k, v, kern = to_dev(k0), to_dev(v0), to_dev(kern0)
        lib().commit(to_dev(dk), to_dev(dv), to_dev(path), to_dev(m), k, v, kern, to_dev(kv), p)
        torch.cuda.synchronize()
        assert lib().sync_status() == 0
        kr, vr = spec_ref.commit(dk, dv, path, m, k0, v0, kv)
        assert np.array_equal(bf16_to_np_bits(k), kr) and np.array_equal(bf16_to_np_bits(v), vr)
        want = kern0.copy()
        pooled, _ = oracle.kernel_pool(kr, kv, c, s, M)
        for b in range(B):
            for j in range(M):
                if kv[b] - m[b] < j * s + c <= kv[b]:
                    want[b, :, j] = pooled[b, :, j]
        assert np.array_equal(bf16_to_np_bits(kern), want)


def test_commit_skips_bad_sequences_and_reports(cuda_lib):
    torch = torch_mod()
    L = lib()
    B, n, d, room = 7, 4, 64, 64
    p = dict(block_size=64, kernel_size=4, kernel_stride=2, topk=4, n_init_blocks=1, n_local_blocks=2, dense_len=0)
    ones = torch.ones((B, 1, n, d), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((B, 1, room, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kern = torch.zeros((B, 1, 20, d), dtype=torch.bfloat16, device="cuda")  # room for kernels up to token 42
    path = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B, 1)
    m = torch.tensor([4, 5, -1, 4, 4, 4, 4], dtype=torch.int32, device="cuda")
    kv = torch.tensor([10, 10, 10, 3, 65, 10, 64], dtype=torch.int32, device="cuda")
    path[5, 2] = n
    L.commit(ones, ones, path, m, k, v, kern, kv, p)
    torch.cuda.synchronize()
    assert L.sync_status() == L.ERR_DEVICE_INDEX
    assert float(k[1:].abs().sum()) == 0.0 and float(v[1:].abs().sum()) == 0.0 and float(kern[1:].abs().sum()) == 0.0
    assert float(k[0, 0, 6:10].sum()) == 4 * d and float(k[0].sum()) == 4 * d
    assert float(kern[0, 0, 3, 0]) == 1.0
    assert L.sync_status() == 0


def test_commit_without_kernel_cache(cuda_lib):
    """Caches that hold no kernel yet need no kernel cache; a sequence whose path would complete one is
    skipped and reported."""
    torch = torch_mod()
    L = lib()
    B, n, d, room = 3, 4, 128, 64
    p = dict(block_size=64, kernel_size=32, kernel_stride=16, topk=4, n_init_blocks=1, n_local_blocks=2, dense_len=0)
    draft = torch.arange(1, n + 1, device="cuda", dtype=torch.float32).to(torch.bfloat16)[:, None].expand(B, 2, n, d).contiguous()
    k, v = (torch.zeros((B, 2, room, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    path = torch.tensor([[0, 2, 3, -1]] * B, dtype=torch.int32, device="cuda")
    m = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    L.commit(draft, draft.clone(), path, m, k, v, None, torch.tensor([3, 31, 20], dtype=torch.int32, device="cuda"), p)
    assert L.sync_status() == 0
    for b, end in enumerate((3, 31, 20)):
        for cache in (k, v):
            assert cache[b, :, end - 3:end, 0].tolist() == [[1.0, 3.0, 4.0]] * 2
            assert float(cache[b].sum()) == 8.0 * 2 * d
    k.zero_(), v.zero_()
    L.commit(draft, draft.clone(), path, m, k, v, None, torch.tensor([31, 32, 50], dtype=torch.int32, device="cuda"), p)
    assert L.sync_status() == L.ERR_DEVICE_INDEX
    assert float(k[0].sum()) == 8.0 * 2 * d and float(k[1:].sum()) == float(v[1:].sum()) == 0.0


# ---- the loop as a serving program runs it

def _speculate(seed, steps, graph):
    """Two sequences: ragged prompts into the caches, then tree steps.  Stands in for the model:
    projections of nothing but seeded noise for q, K, V and of the attention's output for the
    target's probabilities.  Returns everything that has to come out alike."""
    torch = torch_mod()
    L = lib()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    bf = torch.bfloat16
    B, Hq, Hkv, d, n, V, room = 2, 32, 2, 128, 12, 501, 700
    p = dict(block_size=64, kernel_size=32, kernel_stride=16, topk=4, n_init_blocks=1, n_local_blocks=2, dense_len=0)
    f, _ = L.rope_freqs(d, 10000.0, "ntk", factor=2.0)
    freqs, rp = f.cuda(), dict(rotary_dim=d)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(bf)  # noqa: E731
    k, v = (torch.zeros((B, Hkv, room, d), dtype=bf, device="cuda") for _ in range(2))
    M = (room - 32) // 16 + 1
    kern = torch.zeros((B, Hkv, M, d), dtype=bf, device="cuda")
    plen = [300, 217]
    cu = torch.tensor([0, 300, 517], dtype=torch.int32, device="cuda")
    kv = torch.tensor(plen, dtype=torch.int32, device="cuda")
    raw = rnd(517, Hq + 2 * Hkv, d)
    qo = torch.empty((517, Hq, d), dtype=bf, device="cuda")
    L.rope_append(raw[:, :Hq], raw[:, Hq:Hq + Hkv], raw[:, Hq + Hkv:], qo, k, v, kv, freqs, rp, cu_q=cu, Tq_max=300)
    L.kernel_pool_varlen(k, kern, kv, cu, 300, p)
    W = torch.randn((Hq * d, V), generator=gen, device="cuda") * 0.05
    x = torch.empty((B, n, Hq + 2 * Hkv, d), dtype=bf, device="cuda")
    q_rot, o = (torch.empty((B, n, Hq, d), dtype=bf, device="cuda") for _ in range(2))
    dk, dv = (torch.empty((B, Hkv, n, d), dtype=bf, device="cuda") for _ in range(2))
    ws = torch.empty(L.workspace_size(L.ENTRY_DECODE, B, n, Hq, Hkv, d, room, p), dtype=torch.uint8, device="cuda")
    target = torch.empty((B, n, V), device="cuda")
    draft = torch.empty((B, n, V), device="cuda")
    tokens = torch.zeros((B, n), dtype=torch.int32, device="cuda")
    u = torch.empty((B, n), device="cuda")
    masks = torch.zeros((B, n), dtype=torch.int64, device="cuda")
    out = _outputs(B, n)

    def step():
        L.rope_drafts(x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], x[..., Hq + Hkv:, :], q_rot, dk, dv, kv, masks, freqs, rp)
        L.decode(q_rot, k, v, kern, kv, o, ws, p, draft_k=dk, draft_v=dv, tree_mask=masks)
        target.copy_(torch.softmax(o.float().view(B * n, Hq * d) @ W, -1).view(B, n, V))
        L.verify(tokens, target, draft, u, out["path"], out["n_path"], out["out_tokens"], tree_mask=masks, kv_len=kv,
                 kv_len_out=kv)
        L.commit(dk, dv, out["path"], out["n_path"], k, v, kern, kv, p)

    rng = np.random.default_rng(seed)
    stream = torch.cuda.Stream()
    captured, log = None, []
    for it in range(steps):
        x.copy_(rnd(B, n, Hq + 2 * Hkv, d))
        parents = [random_tree(rng, n, 2) for _ in range(B)]
        masks.copy_(to_dev(np.array([masks_of(t) for t in parents], dtype=np.uint64)))
        draft.copy_(torch.softmax(torch.randn((B, n, V), generator=gen, device="cuda"), -1))
        pick = torch.multinomial(draft.view(B * n, V), n, replacement=True, generator=gen).view(B, n, n)
        for b in range(B):
            for i in range(1, n):
                tokens[b, i] = pick[b, parents[b][i], i]
        u.copy_(torch.rand((B, n), generator=gen, device="cuda"))
        before = kv.clone()
        torch.cuda.synchronize()
        if graph and captured is None:
            state = [t.clone() for t in (kv, k, v, kern)]
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                step()
            torch.cuda.synchronize()
            for t, s in zip((kv, k, v, kern), state):
                t.copy_(s)
            torch.cuda.synchronize()
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured, stream=stream):
                step()
        if graph:
            with torch.cuda.stream(stream):
                captured.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert L.sync_status() == 0
        for b in range(B):
            path, toks = spec_ref.verify(tokens[b].tolist(), parents[b], target[b].double().cpu().numpy(),
                                         draft[b].double().cpu().numpy(), u[b].cpu().numpy(), True)
            _check(out, b, n, path, toks)
            assert kv[b].item() == before[b].item() + len(path)
            # the committed rows are the drafts' K at their positions: the same bits as a chunk of them gives
            row = x[b, path]
            ck, cv = (torch.zeros((1, Hkv, room, d), dtype=bf, device="cuda") for _ in range(2))
            L.rope_append(row[None, :, :Hq], row[None, :, Hq:Hq + Hkv], row[None, :, Hq + Hkv:],
                          torch.empty((1, len(path), Hq, d), dtype=bf, device="cuda"), ck, cv, kv[b:b + 1].clone(), freqs, rp)
            at = slice(before[b].item(), kv[b].item())
            assert torch.equal(k[b, :, at], ck[0, :, at]) and torch.equal(v[b, :, at], cv[0, :, at])
        log.append({key: t.clone() for key, t in out.items()})
    lens = kv.cpu().numpy()
    pooled, _ = oracle.kernel_pool(bf16_to_np_bits(k), lens, 32, 16, M)
    got = bf16_to_np_bits(kern)
    for b in range(B):
        m = oracle.n_kernels(int(lens[b]), 32, 16)
        assert np.array_equal(got[b, :, :m], pooled[b, :, :m])
    return k, v, kern, kv, log


def test_speculative_loop_eager_and_captured(cuda_lib):
    torch = torch_mod()
    a, b = _speculate(31, 8, False), _speculate(31, 8, True)
    assert all(torch.equal(x, y) for x, y in zip(a[:4], b[:4]))
    assert all(torch.equal(x[key], y[key]) for x, y in zip(a[4], b[4]) for key in x)
    assert int(a[3].sum()) > 517 + 16  # more than the roots alone
