"""The rotary, verification and commit entry points refuse bad arguments on the host, before any
launch, and the binding refuses tensors of other types and shapes -- all without a GPU.  The table
of frequencies is checked against 50-digit arithmetic."""
import ctypes
import math
from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal, getcontext

import pytest

from block_sparse_long_infllm_gb300 import infllmv2 as L

P = dict(block_size=64, kernel_size=32, kernel_stride=16, topk=64, n_init_blocks=1, n_local_blocks=2, dense_len=8192)
INV, UNS = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED


def at(i):  # never dereferenced: every call here is refused first
    return ctypes.c_void_p((1 << 32) + (i << 28))


def rp(**kw):
    return ctypes.byref(L.RopeParams.make(dict(dict(rotary_dim=128, interleaved=0, attn_scale=1.0), **kw)))


def rope_args(**kw):
    a = dict(q=at(1), ld_q=4096, k=at(2), ld_k=256, pos=at(3), freqs=at(4), rows=8, Hq=32, Hk=2, d=128, dtype=0,
             transposed=0, q_out=at(5), ld_qo=4096, k_out=at(6), ld_ko=256, rope=rp(), stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(rope=rp(rotary_dim=0)), INV), (dict(rope=rp(rotary_dim=7)), INV), (dict(rope=rp(rotary_dim=130)), INV),
    (dict(rope=rp(interleaved=2)), INV), (dict(rope=rp(attn_scale=-1.0)), INV),
    (dict(rope=rp(attn_scale=float("nan"))), INV), (dict(rope=None), INV), (dict(d=96), UNS), (dict(dtype=2), UNS),
    (dict(rows=-1), INV), (dict(rows=(1 << 30) + 1), INV), (dict(Hq=0), INV), (dict(Hk=-1), INV), (dict(q=None), INV),
    (dict(pos=None), INV),
    (dict(freqs=None), INV), (dict(q_out=None), INV), (dict(k=None), INV), (dict(k_out=None), INV), (dict(Hk=0), INV),
    (dict(ld_q=4095), INV), (dict(ld_ko=255), INV), (dict(q=ctypes.c_void_p((1 << 32) + 8)), INV),
    (dict(freqs=ctypes.c_void_p((1 << 32) + 4)), INV),
    (dict(q_out=at(1), ld_qo=8192), INV),                                    # in place with another stride
    (dict(q_out=ctypes.c_void_p((1 << 32) + (1 << 28) + 256)), INV),         # shifted by one head
    (dict(k_out=at(5)), INV), (dict(k_out=at(1)), INV), (dict(q_out=at(2)), INV),
])
def test_rope_refuses(built_lib, kw, code):
    assert built_lib.infllmv2_rope(*rope_args(**kw)) == code


def test_rope_without_rows_is_a_noop(built_lib):
    assert built_lib.infllmv2_rope(*rope_args(rows=0, q=None)) == L.OK


def append_args(**kw):
    a = dict(q=at(1), ld_q=4096, k=at(2), ld_k=256, v=at(3), ld_v=256, q_out=at(4), kc=at(5), vc=at(6), kv=at(7),
             cu=None, freqs=at(8), B=2, Tq=8, total=16, Hq=32, Hkv=2, d=128, L_max=64, rope=rp(), stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(d=80), UNS), (dict(Hq=6, total=16), UNS), (dict(Hq=33), INV), (dict(Tq=65, total=130), INV),
    (dict(total=17), INV), (dict(total=-1, cu=at(9)), INV), (dict(total=(1 << 30) + 1, cu=at(9)), INV), (dict(L_max=0), INV), (dict(L_max=(1 << 28) + 1), INV),
    (dict(B=-1), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(q_out=None), INV),
    (dict(kc=None), INV), (dict(vc=None), INV), (dict(kv=None), INV), (dict(freqs=None), INV), (dict(ld_k=128), INV),
    (dict(q_out=at(1), ld_q=8192), INV), (dict(q_out=at(2)), INV), (dict(cu=ctypes.c_void_p((1 << 32) + 2)), INV),
    (dict(rope=rp(rotary_dim=129)), INV),
])
def test_rope_append_refuses(built_lib, kw, code):
    assert built_lib.infllmv2_rope_append(*append_args(**kw)) == code


def test_rope_append_without_tokens_is_a_noop(built_lib):
    assert built_lib.infllmv2_rope_append(*append_args(B=0)) == L.OK
    assert built_lib.infllmv2_rope_append(*append_args(Tq=0, total=0)) == L.OK
    assert built_lib.infllmv2_rope_append(*append_args(cu=at(9), total=0)) == L.OK


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), UNS), (dict(d=32), UNS), (dict(total=3), INV), (dict(dq=None), INV), (dict(dk=None), INV),
    (dict(dvo=None), INV), (dict(kv=None), INV), (dict(ld_dq=100), INV),
    (dict(dqo=at(1), dtype=0), INV),                       # bf16 over its own fp32 input
    (dict(dqo=at(1), dtype=1, ld_dq=8192), INV), (dict(dko=at(4)), INV), (dict(dvo=at(5)), INV),
])
def test_rope_append_bwd_refuses(built_lib, kw, code):
    a = dict(dq=at(1), dk=at(2), dv=at(3), dqo=at(4), ld_dq=4096, dko=at(5), ld_dk=256, dvo=at(6), ld_dv=256, kv=at(7),
             cu=None, freqs=at(8), B=2, Tq=8, total=16, Hq=32, Hkv=2, d=128, L_max=64, dtype=1, rope=rp(), stream=None)
    a.update(kw)
    assert built_lib.infllmv2_rope_append_bwd(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=65), UNS), (dict(n=-1), INV), (dict(mask=None), INV), (dict(mask=ctypes.c_void_p((1 << 32) + 4)), INV),
    (dict(dk=None), INV), (dict(q=None), INV), (dict(kv=None), INV), (dict(d=256), UNS), (dict(q_out=at(3)), INV),
])
def test_rope_drafts_refuses(built_lib, kw, code):
    a = dict(q=at(1), ld_q=4096, k=at(2), ld_k=256, v=at(3), ld_v=256, q_out=at(4), dk=at(5), dv=at(6), kv=at(7),
             mask=at(8), freqs=at(9), B=2, n=8, Hq=32, Hkv=2, d=128, rope=rp(), stream=None)
    a.update(kw)
    assert built_lib.infllmv2_rope_drafts(*a.values()) == code


def verify_args(**kw):
    a = dict(tokens=at(1), mask=at(2), nodes=None, target=at(3), draft=at(4), u=at(5), kv=None, B=2, n=8, V=1000, dtype=1,
             replace=1, path=at(6), n_path=at(7), out=at(8), kv_out=None, stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(n=65), UNS), (dict(n=-1), INV), (dict(V=0), INV), (dict(V=(1 << 24) + 1), UNS), (dict(dtype=2), UNS),
    (dict(tokens=None), INV), (dict(target=None), INV), (dict(u=None), INV), (dict(path=None), INV),
    (dict(n_path=None), INV), (dict(out=None), INV), (dict(kv=at(9)), INV), (dict(kv_out=at(9)), INV),
    (dict(target=ctypes.c_void_p((1 << 32) + 4)), INV), (dict(draft=ctypes.c_void_p((1 << 32) + 8)), INV),
    (dict(mask=ctypes.c_void_p((1 << 32) + 4)), INV), (dict(B=-1), INV),
])
def test_verify_refuses(built_lib, kw, code):
    assert built_lib.infllmv2_verify(*verify_args(**kw)) == code


def test_verify_without_work_is_a_noop(built_lib):
    assert built_lib.infllmv2_verify(*verify_args(B=0)) == L.OK
    assert built_lib.infllmv2_verify(*verify_args(n=0)) == L.OK


@pytest.mark.parametrize("kw,code", [
    (dict(n=65), UNS), (dict(d=96), UNS), (dict(Hkv=0), INV), (dict(L_max=0), INV), (dict(M_max=-1), INV),
    (dict(dk=None), INV), (dict(path=None), INV), (dict(n_path=None), INV), (dict(kv=None), INV),
    (dict(kern=None), INV), (dict(kc=ctypes.c_void_p((1 << 32) + 4)), INV), (dict(params=None), INV),
    (dict(params=ctypes.byref(L.Params.make(dict(P, kernel_stride=0)))), INV),
])
def test_commit_refuses(built_lib, kw, code):
    a = dict(dk=at(1), dv=at(2), path=at(3), n_path=at(4), kc=at(5), vc=at(6), kern=at(7), kv=at(8), B=2, n=8, Hkv=2,
             d=128, L_max=64, M_max=3, params=ctypes.byref(L.Params.make(P)), stream=None)
    a.update(kw)
    assert built_lib.infllmv2_commit(*a.values()) == code


# ---- the table of frequencies

def _pi():
    getcontext().prec = 50
    return Decimal("3.14159265358979323846264338327950288419716939937510")


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (96, 1e6)])
def test_freqs_match_50_digits(built_lib, rot, base):
    freqs, scale = L.rope_freqs(rot, base)
    two_pi = 2 * _pi()
    assert scale == 1.0
    for i, f in enumerate(freqs.tolist()):
        turns = (Decimal(base).ln() * Decimal(-2 * i) / Decimal(rot)).exp() / two_pi
        # pow within 1 ulp (2^-52 of the value), the division and the cut to 2^-64 beside it
        assert abs(Decimal(f % (1 << 64)) / Decimal(1 << 64) - turns) <= turns * Decimal(2) ** -50 + Decimal(2) ** -63


def test_freqs_scalings(built_lib):
    import torch
    rot, base, s, L0 = 64, 10000.0, 8.0, 4096
    plain = L.rope_freqs(rot, base)[0].double()
    lin, m = L.rope_freqs(rot, base, "linear", factor=s)
    assert m == 1.0 and torch.allclose(lin.double() * s, plain, rtol=2 ** -40)
    ntk, m = L.rope_freqs(rot, base, "ntk", factor=s)
    assert m == 1.0 and torch.allclose(ntk.double(), L.rope_freqs(rot, base * s ** (rot / (rot - 2)))[0].double(), rtol=2 ** -40)
    assert torch.allclose(ntk[-1].double() * s, plain[-1], rtol=2 ** -40)  # the slowest pair is slowed by the factor
    yarn, m = L.rope_freqs(rot, base, "yarn", factor=s, orig_len=L0)
    assert abs(m - 1.2079441541679836) < 1e-7
    turns = L0 * plain / 2.0 ** 64
    ratio = plain / yarn.double()
    assert torch.allclose(ratio[turns > 40], torch.ones(1, dtype=torch.float64), rtol=2 ** -40)
    assert torch.allclose(ratio[turns < 0.7], torch.full((1,), s, dtype=torch.float64), rtol=2 ** -40)
    assert bool((ratio[1:] >= ratio[:-1] - 1e-9).all())
    div = torch.linspace(1.0, 30.0, rot // 2)
    lng, m = L.rope_freqs(rot, base, "divisors", factor=s, orig_len=L0, divisors=div)
    assert torch.allclose(lng.double() * div.double(), plain, rtol=2 ** -40)
    assert abs(m - 1.1180339887498949) < 1e-6  # sqrt(1 + ln 8 / ln 4096) = sqrt(1.25)


@pytest.mark.parametrize("rot,base,s,L0,fast,slow", [
    (64, 10000.0, 8.0, 4096, 32.0, 1.0), (128, 10000.0, 4.0, 32768, 32.0, 1.0), (128, 500000.0, 16.0, 8192, 32.0, 1.0),
    (96, 1e6, 2.0, 2048, 16.0, 2.0), (32, 10000.0, 40.0, 4096, 64.0, 0.5), (64, 10000.0, 8.0, 128, 32.0, 1.0)])
def test_freqs_yarn_between_its_ends(built_lib, rot, base, s, L0, fast, slow):
    """Every pair against the formula in 50 digits: the ramp over i runs from the pair (rounded down) that turns
    beta_fast times within orig_len tokens to the one (rounded up) that turns beta_slow times."""
    _pi()
    D = Decimal
    two_pi = 2 * _pi()

    def pair(turns):
        return D(rot) * (D(L0) / (D(turns) * two_pi)).ln() / (2 * D(base).ln())

    low = max(int(pair(fast).to_integral_value(ROUND_FLOOR)), 0)
    high = min(int(pair(slow).to_integral_value(ROUND_CEILING)), rot - 1)
    freqs, scale = L.rope_freqs(rot, base, "yarn", factor=s, orig_len=L0, beta_fast=fast, beta_slow=slow)
    assert abs(scale - (0.1 * math.log(s) + 1)) <= 2 ** -23
    between = 0
    for i, f in enumerate(freqs.tolist()):
        theta = (D(base).ln() * D(-2 * i) / D(rot)).exp()
        ramp = min(max(D(i - low) / D(high - low), D(0)), D(1))
        turns = (theta / D(s) * ramp + theta * (1 - ramp)) / two_pi
        between += 0 < ramp < 1
        # fp64: pow within 1 ulp, then a handful of operations, and the cut to 2^-64
        assert abs(D(f % (1 << 64)) / D(1 << 64) - turns) <= turns * D(2) ** -48 + D(2) ** -63, i
    assert between >= 3


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(base=1.0), dict(base=float("nan")), dict(scaling="linear", factor=0.0),
    dict(scaling="ntk", factor=float("inf")), dict(scaling="ntk", rotary_dim=2, factor=2.0),
    dict(scaling="yarn", factor=2.0, orig_len=0), dict(scaling="yarn", factor=2.0, orig_len=64, beta_slow=40.0),
    dict(scaling="divisors", factor=2.0, orig_len=64), dict(scaling="ntk", factor=1e-320),
    dict(scaling="ntk", factor=1e308), dict(scaling="linear", factor=1e-320),
    dict(scaling="divisors", factor=2.0, orig_len=64, rotary_dim=4, divisors=[1.0, 0.0]),
])
def test_freqs_refuse(built_lib, kw):
    with pytest.raises(L.InfLLMv2Error):
        L.rope_freqs(**dict(dict(rotary_dim=64, base=10000.0), **kw))


def test_freqs_refuse_names_and_sizes(built_lib):
    with pytest.raises(ValueError):
        L.rope_freqs(64, scaling="cubic")
    with pytest.raises(ValueError):
        L.rope_freqs(64, scaling="divisors", factor=2.0, orig_len=64, divisors=[1.0] * 31)


# ---- the binding's own checks (CPU tensors stand in: types and shapes are looked at first)

def _tensors():
    import torch
    bf = torch.bfloat16
    B, T, Hq, Hkv, d, Lm, n, V = 2, 4, 4, 2, 64, 32, 4, 10
    i32 = torch.int32
    return dict(
        rope=dict(q=torch.zeros(T, Hq, d, dtype=bf), k=torch.zeros(T, Hkv, d, dtype=bf), pos=torch.zeros(T, dtype=i32),
                  q_out=torch.zeros(T, Hq, d, dtype=bf), k_out=torch.zeros(T, Hkv, d, dtype=bf),
                  freqs=torch.zeros(32, dtype=torch.int64), rope=dict(rotary_dim=64)),
        rope_append=dict(q=torch.zeros(B, T, Hq, d, dtype=bf), k_new=torch.zeros(B, T, Hkv, d, dtype=bf),
                         v_new=torch.zeros(B, T, Hkv, d, dtype=bf), q_out=torch.zeros(B, T, Hq, d, dtype=bf),
                         k_cache=torch.zeros(B, Hkv, Lm, d, dtype=bf), v_cache=torch.zeros(B, Hkv, Lm, d, dtype=bf),
                         kv_len=torch.zeros(B, dtype=i32), freqs=torch.zeros(32, dtype=torch.int64),
                         rope=dict(rotary_dim=64)),
        rope_append_bwd=dict(dq=torch.zeros(B, T, Hq, d), dk=torch.zeros(B, Hkv, Lm, d), dv=torch.zeros(B, Hkv, Lm, d),
                             dq_out=torch.zeros(B, T, Hq, d, dtype=bf), dk_out=torch.zeros(B, T, Hkv, d, dtype=bf),
                             dv_out=torch.zeros(B, T, Hkv, d, dtype=bf), kv_len=torch.zeros(B, dtype=i32),
                             freqs=torch.zeros(32, dtype=torch.int64), rope=dict(rotary_dim=64)),
        rope_drafts=dict(q=torch.zeros(B, n, Hq, d, dtype=bf), k_new=torch.zeros(B, n, Hkv, d, dtype=bf),
                         v_new=torch.zeros(B, n, Hkv, d, dtype=bf), q_out=torch.zeros(B, n, Hq, d, dtype=bf),
                         draft_k=torch.zeros(B, Hkv, n, d, dtype=bf), draft_v=torch.zeros(B, Hkv, n, d, dtype=bf),
                         kv_len=torch.zeros(B, dtype=i32), tree_mask=torch.zeros(B, n, dtype=torch.int64),
                         freqs=torch.zeros(32, dtype=torch.int64), rope=dict(rotary_dim=64)),
        verify=dict(tokens=torch.zeros(B, n, dtype=i32), target=torch.zeros(B, n, V), draft=torch.zeros(B, n, V),
                    u=torch.zeros(B, n), path=torch.zeros(B, n, dtype=i32), n_path=torch.zeros(B, dtype=i32),
                    out_tokens=torch.zeros(B, n, dtype=i32), tree_mask=torch.zeros(B, n, dtype=torch.int64),
                    n_nodes=torch.zeros(B, dtype=i32), kv_len=torch.zeros(B, dtype=i32),
                    kv_len_out=torch.zeros(B, dtype=i32)),
        commit=dict(draft_k=torch.zeros(B, Hkv, n, d, dtype=bf), draft_v=torch.zeros(B, Hkv, n, d, dtype=bf),
                    path=torch.zeros(B, n, dtype=i32), n_path=torch.zeros(B, dtype=i32),
                    k_cache=torch.zeros(B, Hkv, Lm, d, dtype=bf), v_cache=torch.zeros(B, Hkv, Lm, d, dtype=bf),
                    kernel_cache=torch.zeros(B, Hkv, 1, d, dtype=bf), kv_len=torch.zeros(B, dtype=i32), params=P))


@pytest.mark.parametrize("name", ["rope", "rope_append", "rope_append_bwd", "rope_drafts", "verify", "commit"])
def test_binding_refuses_types_shapes_and_cpu_tensors(built_lib, name):
    import torch
    args, fn = _tensors()[name], getattr(L, name)
    with pytest.raises(ValueError, match="CUDA device"):
        fn(**args)
    for key, t in args.items():
        if not isinstance(t, torch.Tensor):
            continue
        for other in (t.to(torch.float64), t[..., :-1], t.flatten()[:-1]):
            with pytest.raises((ValueError, IndexError)) as e:
                fn(**dict(args, **{key: other}))
            assert "CUDA device" not in str(e.value), (key, other.shape)
    with pytest.raises(TypeError):
        fn(**dict(args, unknown=1))


def test_binding_takes_fused_slices_and_refuses_uneven_rows(built_lib):
    import torch
    bf = torch.bfloat16

    def call(q, B, T):
        a = _tensors()["rope_append"]
        new = lambda h: torch.zeros(B, T, h, 64, dtype=bf)  # noqa: E731
        a.update(q=q, k_new=new(2), v_new=new(2), q_out=torch.zeros(q.shape, dtype=bf), k_cache=torch.zeros(B, 2, 32, 64, dtype=bf),
                 v_cache=torch.zeros(B, 2, 32, 64, dtype=bf), kv_len=torch.zeros(B, dtype=torch.int32))
        L.rope_append(**a)

    x = torch.zeros(2, 4, 8, 64, dtype=bf)
    for q in (x[..., :4, :], x[:, :1, 4:], x[:1, :1, 4:], x[:, :, :1], x[:1]):  # all checks but the device's pass
        with pytest.raises(ValueError, match="CUDA device"):
            call(q, *q.shape[:2])
    for q in (x[:, :3], x[..., ::2, :], x.transpose(0, 1), x.expand(2, 4, 8, 64)[:, :, :1].expand(2, 4, 8, 64)):
        with pytest.raises(ValueError, match="evenly spaced|dense heads"):
            call(q, *q.shape[:2])


def test_binding_takes_parameters_as_dicts_and_structures(built_lib):
    a = _tensors()
    for rope in (dict(rotary_dim=64), L.RopeParams.make(dict(rotary_dim=64, interleaved=1, attn_scale=1.5))):
        with pytest.raises(ValueError, match="CUDA device"):
            L.rope(**dict(a["rope"], rope=rope))
    with pytest.raises(ValueError, match="CUDA device"):
        L.commit(**dict(a["commit"], params=L.Params.make(P)))
    with pytest.raises(KeyError):
        L.rope(**dict(a["rope"], rope=dict(interleaved=1)))
    with pytest.raises(ValueError, match="parameter structure"):
        L.rope(**dict(a["rope"], rope=L.Params.make(P)))
    with pytest.raises(ValueError, match="freqs"):
        L.rope(**dict(a["rope"], rope=dict(rotary_dim=32)))


def test_verification_waits_are_decided_by_whole_warps():
    """A lane that gives up a bounded wait alone parts its warp, and the other lanes' full-mask shuffles
    behind the wait have no defined end.  (A wait that runs out cannot be provoked by a valid call.)"""
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_long_infllm_gb300",
                        "csrc", "verify.cu")
    text = re.sub(r"//[^\n]*", "", open(path).read())
    waits = [text[max(m.start() - 40, 0):m.start()] for m in re.finditer(r"\bmbar_(try_|test_)?wait\(", text)]
    assert waits and all(w.rstrip().endswith("__all_sync(0xffffffffu,") for w in waits)
