"""Rotary positions on the GPU against the definition in fp64: alone (both pair layouts, parts of the
head, bf16 and fp32, far and negative positions, strided rows, in place), transposed (the gradient),
into the caches and back, and of draft trees; then the chunk path as a training step runs it, against
autograd of the same chain in fp64."""
import math

import numpy as np
import pytest

from spec_ref import masks_of, random_tree, rope_tolerance, rotate, turn_fraction

from harness import lib, torch_mod

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _dt(name):
    torch = torch_mod()
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rand(rng, shape, dtype):
    torch = torch_mod()
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, ref, amp, half, what):
    err = np.abs(_np(got) - ref)
    tol = rope_tolerance(ref, amp, half)
    assert np.all(err <= tol), f"{what}: worst {np.max(err / tol):.2f} of the tolerance"


def _freqs(rot, base=10000.0, **kw):
    f, scale = lib().rope_freqs(rot, base, **kw)
    return f.cuda(), f.numpy().view(np.uint64), scale


def _status():
    torch_mod().cuda.synchronize()
    return lib().sync_status()


@pytest.mark.parametrize("rows,Hq,Hk,d,rot,inter,dtype", [
    (1, 1, 1, 64, 64, 0, "bf16"), (1, 32, 2, 128, 128, 0, "bf16"), (3, 32, 2, 128, 128, 1, "bf16"),
    (7, 5, 3, 64, 32, 0, "bf16"), (33, 2, 1, 64, 16, 1, "fp32"), (65, 16, 16, 128, 96, 0, "fp32"),
    (130, 4, 0, 128, 2, 0, "bf16"), (130, 3, 1, 128, 50, 1, "bf16"), (130, 3, 1, 64, 6, 0, "fp32"),
    (700, 33, 1, 64, 64, 1, "fp32"), (1301, 3, 1, 128, 64, 0, "bf16"), (1301, 7, 2, 128, 126, 0, "fp32"),
    (2601, 2, 1, 64, 32, 1, "bf16"), (2601, 1, 1, 64, 64, 0, "fp32"), (4999, 1, 1, 128, 128, 0, "bf16")])
@pytest.mark.parametrize("transposed", [False, True])
def test_rope_matches_definition(cuda_lib, rows, Hq, Hk, d, rot, inter, dtype, transposed):
    torch = torch_mod()
    rng = np.random.default_rng(rows * 7 + rot)
    t = _dt(dtype)
    q = _rand(rng, (rows, Hq, d), t)
    k = _rand(rng, (rows, Hk, d), t) if Hk else None
    pos = rng.integers(0, 200000, rows).astype(np.int32)
    pos[0] = 0
    dev, table, scale = _freqs(rot, 10000.0, scaling="yarn", factor=4.0, orig_len=4096)
    qo = torch.full_like(q, float("nan"))
    ko = torch.full_like(k, float("nan")) if Hk else None
    lib().rope(q, k, torch.from_numpy(pos).cuda(), qo, ko, dev, dict(rotary_dim=rot, interleaved=inter, attn_scale=scale),
               transposed=transposed)
    assert _status() == 0
    angle = turn_fraction(table, pos)
    for got, x in ((qo, q), (ko, k)):
        if x is None:
            continue
        ref, amp = rotate(_np(x), angle, rot, bool(inter), scale, transposed)
        _close(got, ref, amp, HALF[dtype], "rows")
        assert torch.equal(got[..., rot:], x[..., rot:])  # the rest of a head is copied


def test_rope_far_and_negative_positions(cuda_lib):
    torch = torch_mod()
    rng = np.random.default_rng(5)
    pos = np.array([0, 1, -1, 2 ** 20 + 1, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31, -123456789], dtype=np.int32)
    q = _rand(rng, (len(pos), 2, 128), torch.float32)
    dev, table, _ = _freqs(128)
    out = torch.empty_like(q)
    lib().rope(q, None, torch.from_numpy(pos).cuda(), out, None, dev, dict(rotary_dim=128))
    assert _status() == 0
    ref, amp = rotate(_np(q), turn_fraction(table, pos), 128, False)
    _close(out, ref, amp, HALF["fp32"], "far positions")


@pytest.mark.parametrize("rot", [64, 20])
def test_rope_in_place_on_a_fused_projection(cuda_lib, rot):
    """q and k are slices of [rows, (Hq + 2 Hkv) d]; they turn where they lie and v stays."""
    torch = torch_mod()
    rng = np.random.default_rng(9)
    rows, Hq, Hkv, d = 19, 8, 2, 64
    x = _rand(rng, (rows, Hq + 2 * Hkv, d), torch.bfloat16)
    before = x.clone()
    pos = np.arange(1000, 1000 + rows, dtype=np.int32)
    dev, table, _ = _freqs(rot)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    lib().rope(q, k, torch.from_numpy(pos).cuda(), q, k, dev, dict(rotary_dim=rot))
    assert _status() == 0
    ref, amp = rotate(_np(before[:, :Hq + Hkv]), turn_fraction(table, pos), rot, False)
    _close(x[:, :Hq + Hkv], ref, amp, HALF["bf16"], "in place")
    assert torch.equal(x[:, Hq + Hkv:], before[:, Hq + Hkv:])


@pytest.mark.parametrize("rot", [64, 20])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rope_takes_rows_off_a_vectors_boundary(cuda_lib, rot, inter, dtype):
    """Row strides that are no multiple of 16 bytes."""
    torch = torch_mod()
    rng = np.random.default_rng(rot)
    rows, H, d, t = 37, 3, 64, _dt(dtype)
    ld = H * d + (3 if dtype == "bf16" else 1)
    x = _rand(rng, (rows, ld), t)
    q = x[:, :H * d].unflatten(1, (H, d))
    before = x.clone()
    pos = np.arange(rows, dtype=np.int32) * 77
    dev, table, _ = _freqs(rot)
    lib().rope(q, None, torch.from_numpy(pos).cuda(), q, None, dev, dict(rotary_dim=rot, interleaved=inter))
    assert _status() == 0
    ref, amp = rotate(_np(before[:, :H * d].unflatten(1, (H, d))), turn_fraction(table, pos), rot, bool(inter))
    _close(q, ref, amp, HALF[dtype], "odd strides")
    assert torch.equal(x[:, H * d:], before[:, H * d:])


@pytest.mark.parametrize("rot,inter", [(16, 0), (10, 0), (10, 1), (2, 0)])
def test_rope_keeps_what_it_copies_bit_for_bit(cuda_lib, rot, inter):
    """NaN payloads and infinities behind the rotated part."""
    torch = torch_mod()
    bits = torch.arange(-32768, 32768, 1, dtype=torch.int32).to(torch.int16).cuda()  # every 16-bit pattern
    q = bits.view(-1, 1, 64).view(torch.bfloat16).clone()
    out = torch.zeros_like(q)
    dev, _, _ = _freqs(rot)
    pos = torch.zeros(q.shape[0], dtype=torch.int32, device="cuda")
    lib().rope(q, None, pos, out, None, dev, dict(rotary_dim=rot, interleaved=inter))
    assert _status() == 0
    assert torch.equal(out.view(torch.int16)[..., rot:], q.view(torch.int16)[..., rot:])


def test_rope_transposed_is_the_gradient(cuda_lib):
    """<R x, g> = <x, R^T g> for both layouts (the operator is linear, so this is its gradient and
    every difference quotient of it), and R^T R = scale^2 on the rotated part."""
    torch = torch_mod()
    rng = np.random.default_rng(3)
    for inter, rot in ((0, 128), (1, 96), (0, 10)):
        x, g = _rand(rng, (50, 4, 128), torch.float32), _rand(rng, (50, 4, 128), torch.float32)
        pos = torch.arange(7000, 7050, dtype=torch.int32, device="cuda")
        dev, _, _ = _freqs(rot)
        rp = dict(rotary_dim=rot, interleaved=inter, attn_scale=1.25)
        y, z, w = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        lib().rope(x, None, pos, y, None, dev, rp)
        lib().rope(g, None, pos, z, None, dev, rp, transposed=True)
        lib().rope(y, None, pos, w, None, dev, rp, transposed=True)
        assert _status() == 0
        lhs, rhs = float((y.double() * g.double()).sum()), float((x.double() * z.double()).sum())
        # each of the 25600 products is off by 2^-21 (|a| + |b|) |g| on either side; |.| < 5 here
        assert abs(lhs - rhs) <= 2 * x.numel() * 2.0 ** -21 * 10 * 5
        want = x.double()
        want[..., :rot] *= 1.25 ** 2
        assert float((w.double() - want).abs().max()) <= 2 * 2.0 ** -21 * 1.25 ** 2 * 4 * float(x.abs().max())


def _chunk(rng, B, Tq, L_max, packed):
    n = [Tq] * B if not packed else [int(v) for v in rng.integers(0, Tq + 1, B)]
    if packed:
        n[0] = Tq
        if B > 2:
            n[1] = 0
    kv = [int(rng.integers(m, L_max + 1)) for m in n]
    return n, np.array(kv, dtype=np.int32)


CHUNKS = [(1, 1, 8, 1, 1, 64, 64, 0, False), (4, 1, 40, 32, 2, 128, 128, 0, False), (3, 37, 100, 4, 2, 64, 32, 1, False),
          (5, 70, 71, 16, 1, 128, 128, 1, True), (7, 301, 512, 2, 2, 64, 64, 0, True), (2, 64, 64, 6, 3, 128, 30, 0, True),
          (9, 5, 33, 8, 8, 64, 14, 1, True), (3, 1201, 1300, 1, 1, 64, 32, 0, True)]


@pytest.mark.parametrize("B,Tq,L_max,Hq,Hkv,d,rot,inter,packed", CHUNKS)
@pytest.mark.parametrize("fused", [False, True])
def test_append_matches_definition(cuda_lib, B, Tq, L_max, Hq, Hkv, d, rot, inter, packed, fused):
    torch = torch_mod()
    rng = np.random.default_rng(B * 100 + Tq)
    n, kv = _chunk(rng, B, Tq, L_max, packed)
    total, behind = sum(n), 3 if packed else 0  # rows behind the last sequence
    rows = total + behind
    bf = torch.bfloat16
    x = _rand(rng, (rows, Hq + 2 * Hkv, d), bf)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    kc, vc = _rand(rng, (B, Hkv, L_max, d), bf), _rand(rng, (B, Hkv, L_max, d), bf)
    kc0, vc0 = kc.clone(), vc.clone()
    qo = torch.full((rows, Hq, d), 7.0, dtype=bf, device="cuda")
    dev, table, _ = _freqs(rot)
    rp = dict(rotary_dim=rot, interleaved=inter)
    cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda") if packed else None
    view = (lambda t: t) if packed else (lambda t: t.unflatten(0, (B, Tq)))
    lib().rope_append(view(q), view(k), view(v), view(qo), kc, vc, torch.from_numpy(kv).cuda(), dev, rp, cu_q=cu,
                      Tq_max=Tq if packed else None)
    assert _status() == 0
    r = 0
    touched = torch.zeros((B, L_max), dtype=torch.bool)
    for b in range(B):
        pos = np.arange(kv[b] - n[b], kv[b])
        angle = turn_fraction(table, pos)
        sl = slice(r, r + n[b])
        ref, amp = rotate(_np(q[sl]), angle, rot, bool(inter))
        _close(qo[sl], ref, amp, HALF["bf16"], "q")
        ref, amp = rotate(_np(k[sl]), angle, rot, bool(inter))
        _close(kc[b, :, kv[b] - n[b]:kv[b]].transpose(0, 1), ref, amp, HALF["bf16"], "k")
        assert torch.equal(vc[b, :, kv[b] - n[b]:kv[b]].transpose(0, 1), v[sl])
        touched[b, kv[b] - n[b]:kv[b]] = True
        r += n[b]
    keep = ~touched[:, None, :, None].cuda()
    assert torch.equal(torch.where(keep, kc, 0), torch.where(keep, kc0, 0))
    assert torch.equal(torch.where(keep, vc, 0), torch.where(keep, vc0, 0))
    assert bool((qo[total:] == 7.0).all())


@pytest.mark.parametrize("B,Tq,L_max,Hq,Hkv,d,rot,inter,packed", CHUNKS)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_append_bwd_matches_definition(cuda_lib, B, Tq, L_max, Hq, Hkv, d, rot, inter, packed, out):
    torch = torch_mod()
    rng = np.random.default_rng(B * 10 + Tq)
    n, kv = _chunk(rng, B, Tq, L_max, packed)
    total = sum(n)
    f32, t = torch.float32, _dt(out)
    dq = _rand(rng, (total, Hq, d), f32)
    dk, dv = _rand(rng, (B, Hkv, L_max, d), f32), _rand(rng, (B, Hkv, L_max, d), f32)
    fused = torch.full((total, Hq + 2 * Hkv, d), 3.0, dtype=t, device="cuda")
    outs = [fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]]
    dev, table, scale = _freqs(rot, 10000.0, scaling="yarn", factor=2.0, orig_len=64)
    rp = dict(rotary_dim=rot, interleaved=inter, attn_scale=scale)
    cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda") if packed else None
    view = (lambda x: x) if packed else (lambda x: x.unflatten(0, (B, Tq)))
    lib().rope_append_bwd(view(dq), dk, dv, *[view(o) for o in outs], torch.from_numpy(kv).cuda(), dev, rp, cu_q=cu,
                          Tq_max=Tq if packed else None)
    assert _status() == 0
    r = 0
    for b in range(B):
        angle = turn_fraction(table, np.arange(kv[b] - n[b], kv[b]))
        sl, x = slice(r, r + n[b]), slice(kv[b] - n[b], kv[b])
        for got, g in ((outs[0][sl], dq[sl]), (outs[1][sl], dk[b, :, x].transpose(0, 1))):
            ref, amp = rotate(_np(g), angle, rot, bool(inter), scale, True)
            _close(got, ref, amp, HALF[out], "gradient")
        assert torch.equal(outs[2][sl], dv[b, :, x].transpose(0, 1).to(t))
        r += n[b]


@pytest.mark.parametrize("rot", [64, 22])
def test_append_bwd_leaves_other_rows_and_turns_in_place(cuda_lib, rot):
    """dq_out is dq; rows of a sequence that is skipped and behind the last one keep what they held."""
    torch = torch_mod()
    rng = np.random.default_rng(rot)
    n, L, H, d = [3, 4, 2], 16, 2, 64
    kv = torch.tensor([3, 17, 9], dtype=torch.int32, device="cuda")  # the second is past the cache
    rows = sum(n) + 2
    dq = _rand(rng, (rows, H, d), torch.float32)
    before = dq.clone()
    dk, dv = _rand(rng, (3, 1, L, d), torch.float32), _rand(rng, (3, 1, L, d), torch.float32)
    ko, vo = (torch.full((rows, 1, d), 7.0, device="cuda") for _ in range(2))
    dev, table, _ = _freqs(rot)
    cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda")
    lib().rope_append_bwd(dq, dk, dv, dq, ko, vo, kv, dev, dict(rotary_dim=rot), cu_q=cu, Tq_max=4)
    assert _status() == lib().ERR_DEVICE_INDEX
    kept = [3, 4, 5, 6, 9, 10]
    assert torch.equal(dq[kept], before[kept]) and bool((ko[kept] == 7.0).all()) and bool((vo[kept] == 7.0).all())
    for sl, x in ((slice(0, 3), np.arange(0, 3)), (slice(7, 9), np.arange(7, 9))):
        ref, amp = rotate(_np(before[sl]), turn_fraction(table, x), rot, False, 1.0, True)
        _close(dq[sl], ref, amp, HALF["fp32"], "dq")
    assert torch.equal(vo[7:9, 0], dv[2, 0, 7:9])


def test_append_skips_bad_sequences_and_reports(cuda_lib):
    torch = torch_mod()
    bf = torch.bfloat16
    B, Tq, L, d = 4, 4, 16, 64
    x = torch.ones((B, Tq, 1, d), dtype=bf, device="cuda")
    kc, vc = torch.zeros((B, 1, L, d), dtype=bf, device="cuda"), torch.zeros((B, 1, L, d), dtype=bf, device="cuda")
    qo = torch.zeros_like(x)
    dev, _, _ = _freqs(64)
    kv = torch.tensor([3, 17, -5, 4], dtype=torch.int32, device="cuda")  # too short, past the cache, negative, fine
    lib().rope_append(x, x.clone(), x.clone(), qo, kc, vc, kv, dev, dict(rotary_dim=64))
    torch.cuda.synchronize()
    assert lib().sync_status() == lib().ERR_DEVICE_INDEX
    assert float(vc[:3].abs().sum()) == 0.0 and float(qo[:3].abs().sum()) == 0.0
    assert float(vc[3, 0, :4].sum()) == 4 * d and float(vc[3, 0, 4:].abs().sum()) == 0.0
    # packed: a length past Tq_max, then descending offsets
    for cu in ([0, 5, 6, 6, 8], [0, 4, 2, 6, 8]):
        kc.zero_(), vc.zero_()
        rows = torch.ones((8, 1, d), dtype=bf, device="cuda")
        lib().rope_append(rows, rows.clone(), rows.clone(), torch.zeros_like(rows), kc, vc,
                          torch.full((B,), 10, dtype=torch.int32, device="cuda"), dev, dict(rotary_dim=64),
                          cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), Tq_max=4)
        torch.cuda.synchronize()
        assert lib().sync_status() == lib().ERR_DEVICE_INDEX
        assert float(vc[3, 0, 8:10].sum()) == 2 * d  # the good last sequence
    assert lib().sync_status() == 0


@pytest.mark.parametrize("B,n,Hq,Hkv,d,rot,inter", [(1, 1, 2, 1, 64, 64, 0), (1, 16, 32, 2, 128, 128, 0),
                                                    (3, 64, 16, 2, 64, 48, 1), (2, 40, 8, 8, 128, 34, 0)])
def test_drafts_match_definition(cuda_lib, B, n, Hq, Hkv, d, rot, inter):
    torch = torch_mod()
    rng = np.random.default_rng(n)
    bf = torch.bfloat16
    x = _rand(rng, (B, n, Hq + 2 * Hkv, d), bf)
    q, k, v = x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], x[..., Hq + Hkv:, :]
    masks = np.array([masks_of(random_tree(rng, n, 3)) for _ in range(B)], dtype=np.uint64)
    masks[-1, -1] = 0  # a place of the tree not in use
    kv = rng.integers(0, 100000, B).astype(np.int32)
    depth = np.array([[max(bin(int(m)).count("1"), 1) for m in row] for row in masks])
    qo = torch.empty((B, n, Hq, d), dtype=bf, device="cuda")
    dk, dv = (torch.empty((B, Hkv, n, d), dtype=bf, device="cuda") for _ in range(2))
    dev, table, _ = _freqs(rot)
    lib().rope_drafts(q, k, v, qo, dk, dv, torch.from_numpy(kv).cuda(), torch.from_numpy(masks.view(np.int64)).cuda(), dev,
                      dict(rotary_dim=rot, interleaved=inter))
    assert _status() == 0
    for b in range(B):
        angle = turn_fraction(table, kv[b] + depth[b] - 1)
        ref, amp = rotate(_np(q[b]), angle, rot, bool(inter))
        _close(qo[b], ref, amp, HALF["bf16"], "q")
        ref, amp = rotate(_np(k[b]), angle, rot, bool(inter))
        _close(dk[b].transpose(0, 1), ref, amp, HALF["bf16"], "k")
        assert torch.equal(dv[b].transpose(0, 1), v[b])


def test_chunk_and_single_steps_give_the_same_bits(cuda_lib):
    """A chunk of T tokens and T decode steps of one token rotate every row alike."""
    torch = torch_mod()
    rng = np.random.default_rng(21)
    bf = torch.bfloat16
    B, T, Hq, Hkv, d, L = 2, 9, 4, 2, 64, 32
    q, k, v = (_rand(rng, (B, T, h, d), bf) for h in (Hq, Hkv, Hkv))
    dev, _, _ = _freqs(64)
    one = [torch.zeros((B, Hkv, L, d), dtype=bf, device="cuda") for _ in range(2)]
    two = [torch.zeros((B, Hkv, L, d), dtype=bf, device="cuda") for _ in range(2)]
    qa, qb = torch.empty_like(q), torch.empty_like(q)
    kv = torch.tensor([T, T + 5], dtype=torch.int32, device="cuda")
    lib().rope_append(q, k, v, qa, *one, kv, dev, dict(rotary_dim=64))
    for t in range(T):
        row = slice(t, t + 1)
        out = torch.empty_like(q[:, row].contiguous())
        lib().rope_append(q[:, row].contiguous(), k[:, row].contiguous(), v[:, row].contiguous(), out, *two,
                          kv - (T - 1 - t), dev, dict(rotary_dim=64))
        qb[:, row] = out
    assert _status() == 0
    assert torch.equal(qa, qb) and torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_training_chunk_matches_fp64_autograd(cuda_lib):
    """rope_append, sparse attention over a selection, its backward and rope_append_bwd, against
    autograd of rotation and masked softmax attention in fp64 on the same bf16 inputs.  Tolerance:
    the attention's own (bf16 weights and outputs: 1e-2 of the largest entry, 5e-3 on average), to
    which the bf16 rounding of the rotated q and K (2^-8 of each score's terms) adds as much."""
    torch = torch_mod()
    L = lib()
    rng = np.random.default_rng(77)
    bf = torch.bfloat16
    B, T, Hq, Hkv, d, rot = 2, 192, 4, 2, 64, 48
    G, bs = Hq // Hkv, 64
    q, k, v = (_rand(rng, (B, T, h, d), bf) for h in (Hq, Hkv, Hkv))
    g = _rand(rng, (B, T, Hq, d), bf)
    p = dict(block_size=bs, kernel_size=32, kernel_stride=16, topk=0, n_init_blocks=1, n_local_blocks=1, dense_len=0)
    dev, table, _ = _freqs(rot)
    rp = dict(rotary_dim=rot)
    kv = torch.full((B,), T, dtype=torch.int32, device="cuda")
    qr = torch.empty_like(q)
    kc, vc = (torch.zeros((B, Hkv, T, d), dtype=bf, device="cuda") for _ in range(2))
    L.rope_append(q, k, v, qr, kc, vc, kv, dev, rp)
    M = (T - 32) // 16 + 1
    kern = torch.zeros((B, Hkv, M, d), dtype=bf, device="cuda")
    L.kernel_pool(kc, kern, 0, T, p)
    S = L.selection_capacity(p, T)
    idx = torch.empty((B, Hkv, T, S), dtype=torch.int32, device="cuda")
    cnt = torch.empty((B, Hkv, T), dtype=torch.int32, device="cuda")
    ws = torch.empty(L.workspace_size(L.ENTRY_BLOCK_SELECT, B, T, Hq, Hkv, d, T, p), dtype=torch.uint8, device="cuda")
    L.block_select(qr, kern, kv, idx, cnt, ws, p, T)
    o, lse = torch.empty_like(q), torch.empty((B, Hq, T), device="cuda")
    L.sparse_attn_fwd(qr, kc, vc, idx, cnt, kv, o, p, lse=lse)
    dq, dk, dv = torch.empty((B, T, Hq, d), device="cuda"), torch.empty((B, Hkv, T, d), device="cuda"), torch.empty((B, Hkv, T, d), device="cuda")
    wb = torch.empty(L.workspace_size(L.ENTRY_SPARSE_ATTN_BWD, B, T, Hq, Hkv, d, T, p), dtype=torch.uint8, device="cuda")
    L.sparse_attn_bwd(qr, kc, vc, o, lse, g, idx, cnt, kv, dq, dk, dv, wb, p)
    gq, gk, gv = (torch.empty((B, T, h, d), device="cuda") for h in (Hq, Hkv, Hkv))
    L.rope_append_bwd(dq, dk, dv, gq, gk, gv, kv, dev, rp)
    assert _status() == 0

    angle = torch.from_numpy(turn_fraction(table, np.arange(T)))
    c, s = angle.cos()[None, :, None], angle.sin()[None, :, None]

    def turn(x):
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat((a * c - b * s, a * s + b * c, x[..., rot:]), -1)

    Q, K, V = (t.double().cpu().requires_grad_(True) for t in (q, k, v))
    t = torch.arange(T)
    block = t // bs
    seen = (t[None] <= t[:, None]) & ((block[None] == 0) | (block[None] == block[:, None]))  # init block and the own one
    sc = torch.einsum("bthd,bxhd->bhtx", turn(Q), turn(K).repeat_interleave(G, 2)) / math.sqrt(d)
    out = torch.einsum("bhtx,bxhd->bthd", sc.masked_fill(~seen, -math.inf).softmax(-1), V.repeat_interleave(G, 2))
    out.backward(g.double().cpu())
    for name, got, want in (("q", gq, Q.grad), ("k", gk, K.grad), ("v", gv, V.grad)):
        err, ref = np.abs(_np(got) - want.numpy()), np.abs(want.numpy())
        assert err.max() <= 2e-2 * ref.max(), f"d{name}: {err.max() / ref.max():.2e}"
        assert err.mean() <= 1e-2 * ref.mean(), f"d{name}: {err.mean() / ref.mean():.2e}"


def test_caches_past_32_bits(cuda_lib):
    """Caches of more than 2^32 elements, written and read back at their far end."""
    torch = torch_mod()
    rng = np.random.default_rng(2)
    bf = torch.bfloat16
    Hkv, d, T = 2, 128, 5
    L = (1 << 24) + 40  # 2 heads of 2^31 elements and more
    dev, table, _ = _freqs(128)
    rp = dict(rotary_dim=128)
    q, k, v = (_rand(rng, (1, T, h, d), bf) for h in (2, Hkv, Hkv))
    kc = torch.zeros((1, Hkv, L, d), dtype=bf, device="cuda")
    vc = torch.zeros((1, Hkv, L, d), dtype=bf, device="cuda")
    kv = torch.tensor([L], dtype=torch.int32, device="cuda")
    qo = torch.empty_like(q)
    lib().rope_append(q, k, v, qo, kc, vc, kv, dev, rp)
    assert _status() == 0
    angle = turn_fraction(table, np.arange(L - T, L))
    ref, amp = rotate(_np(k[0]), angle, 128, False)
    _close(kc[0, :, L - T:].transpose(0, 1), ref, amp, HALF["bf16"], "k")
    assert torch.equal(vc[0, :, L - T:].transpose(0, 1), v[0])
    assert float(vc[0, 1, :T].abs().sum()) == 0.0  # what a wrapped offset would hit
    # the commit of a path at the same end, over the rows just written
    p = dict(block_size=64, kernel_size=32, kernel_stride=16, topk=4, n_init_blocks=1, n_local_blocks=2, dense_len=0)
    kern = torch.zeros((1, Hkv, (L - 32) // 16 + 1, d), dtype=bf, device="cuda")
    dk, dv = _rand(rng, (1, Hkv, 8, d), bf), _rand(rng, (1, Hkv, 8, d), bf)
    path = torch.tensor([[1, 3, 4, 7, -1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    lib().commit(dk, dv, path, torch.tensor([4], dtype=torch.int32, device="cuda"), kc, vc, kern, kv, p)
    assert _status() == 0
    assert torch.equal(kc[0, :, L - 4:], dk[0, :, [1, 3, 4, 7]]) and torch.equal(vc[0, :, L - 4:], dv[0, :, [1, 3, 4, 7]])
    del vc, kern
    # gradients out of caches of the same size
    g = torch.zeros((1, Hkv, L, d), dtype=torch.float32, device="cuda")
    g[0, :, L - T:] = kc[0, :, L - T:].float()
    outs = [torch.empty((1, T, h, d), device="cuda") for h in (2, Hkv, Hkv)]
    lib().rope_append_bwd(torch.zeros((1, T, 2, d), device="cuda"), g, g, *outs, kv, dev, rp)
    assert _status() == 0
    ref, amp = rotate(_np(g[0, :, L - T:].transpose(0, 1)), angle, 128, False, 1.0, True)
    _close(outs[1][0], ref, amp, HALF["fp32"], "dk")
    assert torch.equal(outs[2][0], g[0, :, L - T:].transpose(0, 1))


def test_rope_on_a_given_stream(cuda_lib):
    """The stream as an object and as a handle, and the current one."""
    torch = torch_mod()
    rng = np.random.default_rng(4)
    q = _rand(rng, (64, 4, 64), torch.bfloat16)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    dev, _, _ = _freqs(64)
    want = torch.empty_like(q)
    lib().rope(q, None, pos, want, None, dev, dict(rotary_dim=64))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, None):
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        with torch.cuda.stream(s if stream is None else torch.cuda.current_stream()):
            lib().rope(q, None, pos, out, None, dev, dict(rotary_dim=64), stream=stream)
        s.synchronize()
        assert torch.equal(out, want)
    assert _status() == 0


@pytest.mark.parametrize("cu,taken", [([0, 4, 8], [True, False]), ([0, 4, 2, 6], [None, False, None]),
                                      ([0, 2, 4, 3, 6], [True, None, False, None]), ([2, 4, 6], [True, True]),
                                      ([-2, 2, 6], [False, True]), ([0, 3, 3, 2 ** 31 - 1], [True, False, False])])
def test_packed_sequences_are_taken_whole_or_not_at_all(cuda_lib, cu, taken):
    """Six rows under offsets that reach past them, descend or start elsewhere: a sequence's rows are all
    written or all left as they were, forward and back, and the call reports.  (None: the sequence shares
    rows with another one; at most one of them is taken.)"""
    torch = torch_mod()
    L, bf, B, d, room = lib(), torch.bfloat16, len(cu) - 1, 64, 16
    rows = torch.ones((6, 1, d), dtype=bf, device="cuda")
    kc, vc = (torch.zeros((B, 1, room, d), dtype=bf, device="cuda") for _ in range(2))
    qo = torch.full_like(rows, 7.0)
    kv = torch.full((B,), 10, dtype=torch.int32, device="cuda")
    dev, _, _ = _freqs(64)
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    L.rope_append(rows, rows.clone(), rows.clone(), qo, kc, vc, kv, dev, dict(rotary_dim=64), cu_q=offsets, Tq_max=4)
    assert _status() == L.ERR_DEVICE_INDEX
    g = torch.ones((B, 1, room, d), device="cuda")
    dq = torch.ones((6, 1, d), device="cuda")
    outs = [torch.full((6, 1, d), 7.0, device="cuda") for _ in range(3)]
    L.rope_append_bwd(dq, g, g.clone(), *outs, kv, dev, dict(rotary_dim=64), cu_q=offsets, Tq_max=4)
    assert _status() == L.ERR_DEVICE_INDEX
    written = []
    for b in range(B):
        n, cached = cu[b + 1] - cu[b], (vc[b, 0].float().sum(-1) > 0).tolist()
        if taken[b] or (taken[b] is None and any(cached)):
            assert cached == [10 - n <= x < 10 for x in range(room)], b
            written += range(cu[b], cu[b + 1])
        else:
            assert not any(cached), b
    assert len(written) == len(set(written))
    for r in range(6):
        assert bool((qo[r] == 7.0).all()) == (r not in written)
        assert [bool((o[r] == 7.0).all()) for o in outs] == [r not in written] * 3


@pytest.mark.parametrize("scaling", ["plain", "yarn"])
@pytest.mark.parametrize("inter", [0, 1])
def test_fp32_rows_lose_no_more_than_a_plain_fp32_rotation(cuda_lib, scaling, inter):
    """The mean error of fp32 rows (a bound on the worst one cannot see an angle held in too few bits)
    against fp64, beside that of factors rounded from fp64 and products and sums in fp32.  The kernel
    takes one of two products and the sum without a rounding between, which is worth more than what its
    factors lose: of about five roundings alike it has four and a twentieth."""
    torch = torch_mod()
    rng = np.random.default_rng(12 + inter)
    rows, H, d = 4096, 8, 128
    kw = dict(scaling="yarn", factor=8.0, orig_len=4096) if scaling == "yarn" else {}
    dev, table, scale = _freqs(d, 10000.0, **kw)
    scale = float(np.float32(scale))
    rp = dict(rotary_dim=d, interleaved=inter, attn_scale=scale)
    x = _rand(rng, (rows, H, d), torch.float32)
    pos = rng.integers(0, 32768, rows).astype(np.int32)
    turns = np.multiply.outer(pos.astype(np.int64).view(np.uint64), table)  # modulo 2^64
    angle = torch.from_numpy((turns.astype(np.float64) / 2.0 ** 64 * 2.0 * np.pi)).cuda()[:, None]

    def turn(x, c, s):
        a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :d // 2], x[..., d // 2:])
        y = (a * c - b * s, a * s + b * c)
        return torch.stack(y, -1).flatten(-2) if inter else torch.cat(y, -1)

    def rms(y, ref):
        return float((y.double() - ref).square().mean().sqrt())

    for back in (False, True):
        c, s = angle.cos() * scale, angle.sin() * scale * (-1.0 if back else 1.0)
        ref, plain = turn(x.double(), c, s), turn(x, c.float(), s.float())
        out = torch.empty_like(x)
        lib().rope(x, None, torch.from_numpy(pos).cuda(), out, None, dev, rp, transposed=back)
        assert _status() == 0
        assert rms(out, ref) <= rms(plain, ref)
    # and the gradient out of the caches
    T = 2048
    kv = torch.tensor([30000], dtype=torch.int32, device="cuda")
    at = np.arange(30000 - T, 30000, dtype=np.int64).view(np.uint64)
    angle = torch.from_numpy(np.multiply.outer(at, table).astype(np.float64) / 2.0 ** 64 * 2.0 * np.pi).cuda()[:, None]
    dq = x[:T].clone()
    dk = torch.zeros((1, 1, 30000, d), device="cuda")
    dk[0, 0, 30000 - T:] = x[T:, 0]
    outs = [torch.empty((1, T, h, d), device="cuda") for h in (H, 1, 1)]
    lib().rope_append_bwd(dq[None], dk, dk.clone(), *outs, kv, dev, rp)
    assert _status() == 0
    c, s = angle.cos() * scale, -angle.sin() * scale
    for got, g in ((outs[0][0], dq), (outs[1][0], x[T:, :1])):
        assert rms(got, turn(g.double(), c, s)) <= rms(turn(g, c.float(), s.float()), turn(g.double(), c, s))
