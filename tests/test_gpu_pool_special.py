"""Infinite and NaN keys in the pooling of semantic kernels, by every call that pools: the mean is what
the definition gives (an infinity, or NaN with both infinities or a NaN among the rows), and columns
without them keep the exact mean, bit for bit."""
import numpy as np
import pytest

import oracle
from block_sparse_long_infllm_gb300 import synth

from harness import bf16_to_np_bits, lib, to_dev, torch_mod

pytestmark = pytest.mark.gpu

SPECIAL = np.array([0x7F80, 0xFF80, 0x7FC1, 0xFFFF, 0x7F81], dtype=np.uint16)  # +inf, -inf, NaNs
SIZES = [(64, 64, 1, 1), (128, 64, 32, 16), (64, 64, 17, 5), (128, 64, 33, 7), (64, 128, 128, 64), (128, 128, 65, 16)]


def _keys(rng, shape):
    """Normal keys; every fifth row holds a few values that are no finite numbers, and one column the largest
    finite one throughout."""
    k = synth.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))
    k[..., 5] = 0x7F7F
    for at in np.ndindex(*shape[:-1]):
        if rng.random() < 0.2:
            k[at][rng.choice(shape[-1], 3, replace=False)] = rng.choice(SPECIAL, 3)
    k[..., 0, 0], k[..., 1, 0] = 0x7F80, 0x7F80  # one sign
    k[..., 0, 1], k[..., 1, 1] = 0x7F80, 0xFF80  # both
    return k


def _params(bs, c, s):
    return dict(block_size=bs, kernel_size=c, kernel_stride=s, topk=4, n_init_blocks=1, n_local_blocks=2, dense_len=0)


def _check(kern, k, kv, c, s, first):
    """Kernels from `first[b]` on that the first kv[b] tokens of k complete."""
    B, H, L, d = k.shape
    M = kern.shape[2]
    got = bf16_to_np_bits(kern)
    finite = np.where((k & 0x7F80) == 0x7F80, 0, k).astype(np.uint16)
    exact, _ = oracle.kernel_pool(finite, kv, c, s, M)
    seen = 0
    for b in range(B):
        for j in range(first[b], oracle.n_kernels(int(kv[b]), c, s)):
            with np.errstate(invalid="ignore"):  # signalling NaNs are widened
                mean = synth.bf16_bits_to_f32(k[b, :, j * s:j * s + c]).astype(np.float64).mean(1)
            g = synth.bf16_bits_to_f32(got[b, :, j])
            ok = np.isfinite(mean)
            assert np.array_equal(got[b, :, j][ok], exact[b, :, j][ok]), (b, j)
            assert np.array_equal(np.isnan(g), np.isnan(mean)), (b, j)
            inf = np.isinf(mean)
            assert np.array_equal(g[inf], mean[inf].astype(np.float32)), (b, j)
            seen += int((~ok).sum())
    assert seen > 0


@pytest.mark.parametrize("d,bs,c,s", SIZES)
def test_pool_of_infinite_and_nan_keys(cuda_lib, d, bs, c, s):
    torch = torch_mod()
    L = lib()
    rng = np.random.default_rng(c)
    B, H, n = 2, 2, 300
    k = _keys(rng, (B, H, n, d))
    M = oracle.n_kernels(n, c, s)
    kv = np.full(B, n, dtype=np.int32)
    kern = torch.zeros((B, H, M, d), dtype=torch.bfloat16, device="cuda")
    L.kernel_pool(to_dev(k), kern, 0, n, _params(bs, c, s))
    assert L.sync_status() == 0
    _check(kern, k, kv, c, s, [0, 0])
    two = torch.zeros_like(kern)
    L.kernel_pool_varlen(to_dev(k), two, to_dev(kv), to_dev(np.array([0, 200, 500], dtype=np.int32)), 300, _params(bs, c, s))
    assert L.sync_status() == 0
    _check(two, k, kv, c, s, [max(0, -(-(100 - c + 1) // s)), 0])


@pytest.mark.parametrize("d,bs,c,s", SIZES)
def test_append_and_commit_pool_infinite_and_nan_keys(cuda_lib, d, bs, c, s):
    torch = torch_mod()
    L = lib()
    rng = np.random.default_rng(c + 1)
    B, H, n, m, start = 2, 2, 300, 60, 200  # 60 tokens complete a kernel of every size
    full = _keys(rng, (B, H, n, d))
    v = np.zeros_like(full)
    M = oracle.n_kernels(n, c, s)
    first = [oracle.n_kernels(start, c, s)] * B
    # one token after another
    k, kern = to_dev(full), torch.zeros((B, H, M, d), dtype=torch.bfloat16, device="cuda")
    k[:, :, start:] = 0
    for x in range(start, start + m):
        row = to_dev(full[:, :, x])
        L.append(row, row.clone(), k, to_dev(v), kern, to_dev(np.full(B, x + 1, dtype=np.int32)), _params(bs, c, s))
    assert L.sync_status() == 0
    kv = np.full(B, start + m, dtype=np.int32)
    _check(kern, full, kv, c, s, first)
    # as one path
    k, two = to_dev(full), torch.zeros_like(kern)
    k[:, :, start:] = 0
    path = torch.arange(m, dtype=torch.int32, device="cuda").repeat(B, 1)
    L.commit(to_dev(full[:, :, start:start + m]), to_dev(v[:, :, start:start + m]), path,
             torch.full((B,), m, dtype=torch.int32, device="cuda"), k, to_dev(v), two, to_dev(kv), _params(bs, c, s))
    assert L.sync_status() == 0
    _check(two, full, kv, c, s, first)


def test_decode_step_pools_infinite_and_nan_keys(cuda_lib):
    """The fused step (the attention's own output is not looked at: keys that are no numbers reach it)."""
    torch = torch_mod()
    L = lib()
    rng = np.random.default_rng(3)
    B, H, Hq, d, n, start = 2, 2, 8, 128, 700, 600
    p = _params(64, 32, 16)
    full = _keys(rng, (B, H, n, d))
    k, kern = to_dev(full), torch.zeros((B, H, oracle.n_kernels(n, 32, 16), d), dtype=torch.bfloat16, device="cuda")
    k[:, :, start:] = 0
    L.kernel_pool(k, kern, 0, start, p)
    v = torch.zeros_like(k)
    q = to_dev(synth.f32_to_bf16_bits(rng.standard_normal((B, 1, Hq, d)).astype(np.float32)))
    ws = torch.empty(L.workspace_size(L.ENTRY_DECODE, B, 1, Hq, H, d, n, p), dtype=torch.uint8, device="cuda")
    for x in range(start, start + 40):
        row = to_dev(full[:, :, x])
        L.decode_step(q, row, torch.zeros_like(row), k, v, kern, to_dev(np.full(B, x + 1, dtype=np.int32)),
                      torch.empty_like(q), ws, p)
    assert L.sync_status() == 0
    _check(kern, full, np.full(B, start + 40, dtype=np.int32), 32, 16, [0, 0])
