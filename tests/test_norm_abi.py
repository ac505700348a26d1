"""The norm, constraint and count entry points refuse bad arguments on the host, before any launch, and
the binding refuses tensors of other types and shapes -- all without a GPU."""
import ctypes

import pytest

from block_sparse_long_infllm_gb300 import infllmv2 as L

INV, UNS, WS = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED, L.ERR_WORKSPACE


def at(i, off=0):  # never dereferenced: every call here is refused first
    return ctypes.c_void_p((1 << 32) + (i << 28) + off)


def rp(**kw):
    return ctypes.byref(L.RopeParams.make(dict(dict(rotary_dim=128, interleaved=0, attn_scale=1.0), **kw)))


def norm(eps=1e-6, offset=0.0, dtype=0):
    return ctypes.byref(L.NormParams(eps, offset, dtype))


NORMS = [
    (dict(norm=None), INV), (dict(norm=norm(eps=0.0)), INV), (dict(norm=norm(eps=-1.0)), INV),
    (dict(norm=norm(eps=2.0)), INV), (dict(norm=norm(eps=float("nan"))), INV), (dict(norm=norm(offset=float("inf"))), INV),
    (dict(norm=norm(dtype=2)), UNS), (dict(qw=at(20, 1)), INV), (dict(kw=at(21, 2), norm=norm(dtype=1)), INV),
    (dict(rope=rp(rotary_dim=7)), INV), (dict(rope=None), INV), (dict(d=96), UNS)]


def rows_args(**kw):
    a = dict(q=at(1), ld_q=4096, k=at(2), ld_k=256, pos=at(3), freqs=at(4), rows=8, Hq=32, Hk=2, d=128, dtype=0,
             q_out=at(5), ld_qo=4096, k_out=at(6), ld_ko=256, qw=at(20), kw=at(21), norm=norm(), rope=rp(), stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", NORMS + [
    (dict(dtype=2), UNS), (dict(rows=-1), INV), (dict(q=None), INV), (dict(pos=None), INV), (dict(q_out=None), INV),
    (dict(k=None), INV), (dict(ld_q=4095), INV), (dict(q_out=at(1), ld_qo=8192), INV), (dict(k_out=at(5)), INV)])
def test_norm_rope_refuses(built_lib, kw, code):
    assert built_lib.infllmv2_norm_rope(*rows_args(**kw)) == code


def rows_back_args(**kw):
    a = dict(dq=at(1), ld_dq=4096, dk=at(2), ld_dk=256, q=at(8), ld_q=4096, k=at(9), ld_k=256, pos=at(3), freqs=at(4),
             rows=8, Hq=32, Hk=2, d=128, dtype=0, dq_out=at(5), ld_dqo=4096, dk_out=at(6), ld_dko=256, qw=at(20), kw=at(21),
             dqw=at(22), dkw=at(23), ws=at(24), ws_bytes=1 << 24, norm=norm(), rope=rp(), stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", NORMS + [
    (dict(dq=None), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(dk=None), INV), (dict(ld_q=4095), INV),
    (dict(ld_k=128), INV), (dict(q=at(8, 8)), INV), (dict(dq_out=at(8)), INV), (dict(dk_out=at(8)), INV),
    (dict(dq_out=at(9)), INV), (dict(dqw=at(22, 2)), INV), (dict(dkw=at(22)), INV), (dict(dkw=at(22, 256)), INV),
    (dict(dqw=at(5, 1024)), INV), (dict(dkw=at(6)), INV), (dict(ws=None), WS), (dict(ws_bytes=1000), WS),
    (dict(ws=at(24, 8)), INV)])
def test_norm_rope_bwd_refuses(built_lib, kw, code):
    assert built_lib.infllmv2_norm_rope_bwd(*rows_back_args(**kw)) == code


def append_args(**kw):
    a = dict(q=at(1), ld_q=4096, k=at(2), ld_k=256, v=at(3), ld_v=256, q_out=at(4), kc=at(5), vc=at(6), kv=at(7),
             cu=None, freqs=at(8), B=2, Tq=8, total=16, Hq=32, Hkv=2, d=128, L_max=64, qw=at(20), kw=at(21), norm=norm(),
             rope=rp(), stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", NORMS + [
    (dict(Hq=6), UNS), (dict(Tq=65, total=130), INV), (dict(total=17), INV), (dict(L_max=0), INV), (dict(q=None), INV),
    (dict(kc=None), INV), (dict(kv=None), INV), (dict(q_out=at(2)), INV)])
def test_norm_rope_append_refuses(built_lib, kw, code):
    assert built_lib.infllmv2_norm_rope_append(*append_args(**kw)) == code


def append_back_args(**kw):
    a = dict(dq=at(1), dk=at(2), dv=at(3), q=at(4), ld_q=4096, k=at(5), ld_k=256, dqo=at(6), ld_dq=4096, dko=at(7), ld_dk=256,
             dvo=at(8), ld_dv=256, kv=at(9), cu=None, freqs=at(10), B=2, Tq=8, total=16, Hq=32, Hkv=2, d=128, L_max=64,
             dtype=1, qw=at(20), kw=at(21), dqw=at(22), dkw=at(23), ws=at(24), ws_bytes=1 << 24, norm=norm(), rope=rp(),
             stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", NORMS + [
    (dict(dtype=3), UNS), (dict(total=3), INV), (dict(dq=None), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(ld_q=100), INV), (dict(dqo=at(4)), INV), (dict(dvo=at(4)), INV), (dict(dvo=at(5)), INV),
    (dict(dqo=at(1), dtype=0), INV), (dict(dqw=at(8)), INV), (dict(ws=None), WS), (dict(ws_bytes=4096), WS)])
def test_norm_rope_append_bwd_refuses(built_lib, kw, code):
    assert built_lib.infllmv2_norm_rope_append_bwd(*append_back_args(**kw)) == code


def drafts_args(**kw):
    a = dict(q=at(1), ld_q=4096, k=at(2), ld_k=256, v=at(3), ld_v=256, q_out=at(4), dk=at(5), dv=at(6), kv=at(7), mask=at(8),
             freqs=at(9), B=2, n=16, Hq=32, Hkv=2, d=128, qw=at(20), kw=at(21), norm=norm(), rope=rp(), stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", NORMS + [(dict(n=65), UNS), (dict(mask=None), INV), (dict(dk=None), INV),
                                             (dict(q=None), INV), (dict(B=-1), INV)])
def test_norm_rope_drafts_refuses(built_lib, kw, code):
    assert built_lib.infllmv2_norm_rope_drafts(*drafts_args(**kw)) == code


def test_calls_without_rows_are_noops(built_lib):
    assert built_lib.infllmv2_norm_rope(*rows_args(rows=0, q=None)) == L.OK
    assert built_lib.infllmv2_norm_rope_append(*append_args(B=0)) == L.OK
    assert built_lib.infllmv2_norm_rope_append(*append_args(Tq=0, total=0)) == L.OK
    assert built_lib.infllmv2_norm_rope_drafts(*drafts_args(B=0)) == L.OK


def test_workspace_of_the_gradient(built_lib):
    size = L.workspace_size(L.ENTRY_NORM_ROPE_BWD, 1, 1, 1, 1, 128, 1, None)
    assert size >= 2 * 128 * 4 and L.workspace_size(L.ENTRY_NORM_ROPE_BWD, 1, 1, 1, 1, 64, 1, None) * 2 == size
    assert L.workspace_size(L.ENTRY_NORM_ROPE_BWD, 1, 1, 1, 1, 96, 1, None) == 0
    assert built_lib.infllmv2_norm_rope_bwd(*rows_back_args(ws_bytes=size - 1)) == WS


def constrain_args(**kw):
    a = dict(logits=at(1), ld=1000, tokens=at(2), mask=at(3), nodes=at(4), history=at(5), ld_h=1000, allowed=at(6), ld_a=32,
             bias=at(7), ld_b=1000, controls=at(8), B=4, n=8, V=1000, dtype=1, probs=1, out=at(9), ld_o=1000, out_dtype=1,
             stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INV), (dict(n=-1), INV), (dict(V=0), INV), (dict(n=65), UNS), (dict(V=(1 << 24) + 1), UNS), (dict(dtype=2), UNS),
    (dict(out_dtype=-1), UNS), (dict(B=1 << 16), INV), (dict(logits=None), INV), (dict(out=None), INV), (dict(ld=999), INV),
    (dict(ld_o=999), INV), (dict(ld_h=999), INV), (dict(ld_a=31), INV), (dict(ld_b=1), INV), (dict(tokens=None), INV),
    (dict(logits=at(1, 4)), INV), (dict(history=at(5, 2)), INV), (dict(bias=at(7, 4)), INV), (dict(allowed=at(6, 2)), INV),
    (dict(controls=at(8, 2)), INV), (dict(mask=at(3, 4)), INV), (dict(out=at(1), ld_o=1004), INV),
    (dict(out=at(1), out_dtype=0), INV), (dict(out=at(1, 16)), INV), (dict(out=at(5)), INV), (dict(out=at(7)), INV),
    (dict(out=at(6)), INV)])
def test_constrain_refuses(built_lib, kw, code):
    assert built_lib.infllmv2_constrain(*constrain_args(**kw)) == code


def test_a_lost_warp_leaves_its_cluster_alone():
    """A warp of a cluster whose bounded wait runs out has not seen the others' pairs, so it cannot know how many more of
    its own they wait for, and pairs that they do not wait for would reach CTAs that have ended: it sends, loads and
    writes nothing more, and its CTA stays until its peers are through and what they sent has arrived.  (A wait that
    runs out cannot be provoked by a valid call.)"""
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_long_infllm_gb300",
                        "csrc", "constrain.cu")
    text = re.sub(r"//[^\n]*", "", open(path).read())
    waits = [text[max(m.start() - 40, 0):m.start()] for m in re.finditer(r"\bmbar_(try_|test_)?wait\(", text)]
    assert waits and all(w.rstrip().endswith("__all_sync(kAll,") for w in waits)
    kernel = text[text.index("constrain_kernel("):text.index("cudaError_t launch_kind(")]
    assert len(re.findall(r"st\.async", kernel)) == 1 and kernel.count("bulk_load(") == 1
    exchange = kernel[kernel.index("const auto exchange"):kernel.index("while (row < to) {")]
    sends = exchange[:exchange.index("st.async")]
    assert sends.rstrip().split("if (")[-1].startswith("lane < parts && !lost)")
    assert "if (!lost) wait(bar" in exchange and "if (tid == 0 && !lost) mbar_arrive_expect_tx(" in exchange
    rows = kernel[kernel.index("while (row < to) {"):]
    assert rows.count("fetch();") == 1 and "if (row < to && !lost) fetch();" in rows
    assert rows.count("wait(&full[warp], loads++") == 1 and "if (!lost) wait(&full[warp], loads++" in rows
    lost = rows[rows.rindex("if (lost) {"):]
    stays = [lost.index(x) for x in ("barrier.cluster.arrive", "barrier.cluster.wait", "< kWaitBudgetCycles",
                                     "mbar_wait(&full[warp]")]
    assert stays == sorted(stays)


def count_args(**kw):
    a = dict(tokens=at(1), lens=at(2), cu=None, B=4, T=8, total=0, V=1000, prompt=0, reset=0, history=at(3), ld=1000,
             stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(total=-1), INV), (dict(V=0), INV), (dict(V=(1 << 24) + 1), UNS),
    (dict(B=65536), INV), (dict(tokens=None), INV), (dict(history=None), INV), (dict(history=at(3, 2)), INV),
    (dict(ld=999), INV), (dict(cu=at(4)), INV), (dict(cu=at(4, 2), lens=None), INV), (dict(tokens=at(1, 2)), INV),
    (dict(T=(1 << 30) // 2), INV)])
def test_count_tokens_refuses(built_lib, kw, code):
    assert built_lib.infllmv2_count_tokens(*count_args(**kw)) == code


def test_constraints_without_work_are_noops(built_lib):
    assert built_lib.infllmv2_constrain(*constrain_args(B=0, logits=None)) == L.OK
    assert built_lib.infllmv2_constrain(*constrain_args(n=0)) == L.OK
    assert built_lib.infllmv2_count_tokens(*count_args(B=0, history=None)) == L.OK
    assert built_lib.infllmv2_count_tokens(*count_args(T=0, tokens=None)) == L.OK


def _tensors():
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    B, T, Hq, Hkv, d, Lm, n, V = 2, 4, 4, 2, 64, 32, 4, 40
    freqs, rope = torch.zeros(32, dtype=torch.int64), dict(rotary_dim=64)
    nm = dict(q_weight=torch.ones(d), k_weight=torch.ones(d), eps=1e-5, offset=1.0)
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype)  # noqa: E731
    f32 = torch.float32
    dw = dict(dq_weight=z(d, dtype=f32), dk_weight=z(d, dtype=f32))
    return dict(
        norm_rope=dict(q=z(T, Hq, d), k=z(T, Hkv, d), pos=z(T, dtype=i32), q_out=z(T, Hq, d), k_out=z(T, Hkv, d), freqs=freqs,
                       rope=rope, norm=nm),
        norm_rope_bwd=dict(dq=z(T, Hq, d), dk=z(T, Hkv, d), q=z(T, Hq, d), k=z(T, Hkv, d), pos=z(T, dtype=i32),
                           dq_out=z(T, Hq, d), dk_out=z(T, Hkv, d), **dw, freqs=freqs, rope=rope, norm=nm),
        norm_rope_append=dict(q=z(B, T, Hq, d), k_new=z(B, T, Hkv, d), v_new=z(B, T, Hkv, d), q_out=z(B, T, Hq, d),
                              k_cache=z(B, Hkv, Lm, d), v_cache=z(B, Hkv, Lm, d), kv_len=z(B, dtype=i32), freqs=freqs,
                              rope=rope, norm=nm),
        norm_rope_append_bwd=dict(dq=z(B, T, Hq, d, dtype=f32), dk=z(B, Hkv, Lm, d, dtype=f32),
                                  dv=z(B, Hkv, Lm, d, dtype=f32), q=z(B, T, Hq, d), k_new=z(B, T, Hkv, d),
                                  dq_out=z(B, T, Hq, d), dk_out=z(B, T, Hkv, d), dv_out=z(B, T, Hkv, d), **dw,
                                  kv_len=z(B, dtype=i32), freqs=freqs, rope=rope, norm=nm),
        norm_rope_drafts=dict(q=z(B, n, Hq, d), k_new=z(B, n, Hkv, d), v_new=z(B, n, Hkv, d), q_out=z(B, n, Hq, d),
                              draft_k=z(B, Hkv, n, d), draft_v=z(B, Hkv, n, d), kv_len=z(B, dtype=i32),
                              tree_mask=z(B, n, dtype=torch.int64), freqs=freqs, rope=rope, norm=nm),
        constrain=dict(logits=z(B, n, V), out=z(B, n, V), tokens=z(B, n, dtype=i32), tree_mask=z(B, n, dtype=torch.int64),
                       n_nodes=z(B, dtype=i32), history=z(B, V, dtype=torch.int16), allowed=z(B, n, 2, dtype=i32),
                       bias=z(B, V, dtype=f32), controls=z(B, 4, dtype=f32)),
        count_tokens=dict(tokens=z(B, T, dtype=i32), history=z(B, V, dtype=torch.int16), n_tokens=z(B, dtype=i32)))


@pytest.mark.parametrize("name", ["norm_rope", "norm_rope_bwd", "norm_rope_append", "norm_rope_append_bwd",
                                  "norm_rope_drafts", "constrain", "count_tokens"])
def test_binding_refuses_types_shapes_and_cpu_tensors(built_lib, name):
    import torch
    args, fn = _tensors()[name], getattr(L, name)
    with pytest.raises(ValueError, match="CUDA device"):
        fn(**args)
    for key, t in args.items():
        if not isinstance(t, torch.Tensor):
            continue
        others = [t.to(torch.float64), t[..., :-1], t.flatten()[:-1]]
        if name == "count_tokens" and key != "n_tokens":
            others[1] = t[:1]  # T and V are these tensors' own
        for other in others:
            with pytest.raises((ValueError, IndexError)) as e:
                fn(**dict(args, **{key: other}))
            assert "CUDA device" not in str(e.value), (key, other.shape)
    if "norm" in args:
        for bad in (torch.ones(63), torch.ones(64, dtype=torch.float64), torch.ones(64, dtype=torch.bfloat16),
                    torch.ones(128)[::2], 1.0):
            with pytest.raises(ValueError) as e:
                fn(**dict(args, norm=dict(args["norm"], k_weight=bad)))
            assert "CUDA device" not in str(e.value)
        for good in (dict(), dict(q_weight=None, eps=1e-3), dict(k_weight=torch.ones(64, dtype=torch.bfloat16))):
            with pytest.raises(ValueError, match="CUDA device"):
                fn(**dict(args, norm=good))
    with pytest.raises(TypeError):
        fn(**dict(args, unknown=1))


def test_binding_takes_rows_of_wider_tensors(built_lib):
    import torch
    a = _tensors()["constrain"]
    x = torch.zeros(2, 4, 50)
    for logits in (x[..., :40], x[:, :1, :40], x[:1, :, :40], x[:1, :1, :40]):
        B, n = logits.shape[:2]
        with pytest.raises(ValueError, match="CUDA device"):
            L.constrain(logits, torch.zeros(B, n, 40), history=torch.zeros(B, 60, dtype=torch.int16)[:, :40],
                        bias=torch.zeros(40))
    for logits in (x[:, :3, :40], torch.zeros(2, 4, 80)[..., ::2], x[..., :40].transpose(0, 1),
                   torch.zeros(2, 1, 40).expand(2, 4, 40)):
        with pytest.raises(ValueError, match="evenly spaced"):
            L.constrain(logits, torch.zeros(logits.shape))
    with pytest.raises(ValueError, match="evenly spaced"):
        L.constrain(**dict(a, bias=torch.zeros(1, 40).expand(2, 40)))
    with pytest.raises(ValueError, match="exclude"):
        L.count_tokens(torch.zeros(5, dtype=torch.int32), torch.zeros(2, 40, dtype=torch.int16),
                       n_tokens=torch.zeros(2, dtype=torch.int32), cu=torch.zeros(3, dtype=torch.int32))
