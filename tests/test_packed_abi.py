"""The packed-batch calls without a GPU: sizes, and every argument the C ABI and
the binding refuse before anything is launched."""

import ctypes

import pytest
import torch

import token_phase_swiglu_b200 as fm

A, MIS, MIS4 = 0x100000, 0x100008, 0x100002   # never dereferenced


def rope(**kw):
    a = dict(theta=1e4, rotary_dim=64) | kw
    return fm.FmlpRope(**a)


def append(q8=False, r=None, **kw):
    a = dict(q=A, qs=256, k=A, ks=128, v=A, vs=128, T=4, cu=A, kv=A, B=2, H=4, Hkv=2, D=64, qg=None, kg=None, eps=1e-6,
             qo=0x900000, kc=A, k_s=A, vc=A, v_s=A, n_max=16, ws=A, wsb=256) | kw
    pre = [a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["T"], a["cu"], a["kv"], a["B"], a["H"], a["Hkv"],
           a["D"], ctypes.byref((r or rope())._c), a["qg"], a["kg"], a["eps"], a["qo"]]
    end = [a["n_max"], a["ws"], a["wsb"], None]
    if q8:
        return fm.lib.fmlp_rope_append_q8(*pre, a["kc"], a["k_s"], a["vc"], a["v_s"], *end)
    return fm.lib.fmlp_rope_append(*pre, a["kc"], a["vc"], *end)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad", [
    dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(kv=None), dict(qo=None), dict(kc=None),
    dict(vc=None), dict(ws=None), dict(q=MIS), dict(k=MIS), dict(qo=MIS), dict(kc=MIS), dict(cu=MIS4), dict(kv=MIS4),
    dict(qg=MIS), dict(kg=MIS), dict(D=80), dict(H=0), dict(Hkv=0), dict(H=2000), dict(B=0), dict(B=65537), dict(T=-1),
    dict(T=1 << 25), dict(n_max=0), dict(n_max=1 << 30), dict(wsb=255), dict(qs=248), dict(ks=120), dict(vs=132),
    dict(qg=A, eps=0.0), dict(kg=A, eps=float("nan")), dict(qo=A + 64), dict(qo=A, qs=264), dict(r=rope(rotary_dim=72)),
    dict(r=rope(rotary_dim=80)), dict(r=rope(rotary_dim=-16)), dict(r=rope(theta=0.0)), dict(r=rope(theta=float("inf"))),
    dict(r=rope(amplitude=float("nan"))), dict(r=rope(scaling="linear", factor=0.0)),
    dict(r=rope(scaling="bands", factor=8.0, low=4.0, high=4.0, original_ctx=10)),
    dict(r=rope(scaling="bands", factor=8.0, low=1.0, high=4.0, original_ctx=0)),
    dict(r=rope(scaling="yarn", factor=8.0, low=1.0, high=4.0, original_ctx=10, theta=1.0)),
])
def test_append_refuses(q8, bad):
    assert append(q8, **bad) == fm.FMLP_ERR_INVALID_ARG


def test_append_q8_refuses_its_scales():
    for bad in (dict(k_s=None), dict(v_s=None), dict(k_s=MIS4), dict(v_s=MIS4)):
        assert append(True, **bad) == fm.FMLP_ERR_INVALID_ARG


def test_no_tokens_is_a_noop():
    assert append(T=0, q=None, k=None, v=None, qo=None) == fm.FMLP_OK


def test_unknown_scaling():
    with pytest.raises(ValueError):
        rope(scaling="other")
    r = rope()
    r._c.scaling = 9
    assert append(r=r) == fm.FMLP_ERR_INVALID_ARG


def test_read_back_refuses():
    def read(**kw):
        a = dict(kq=A, ks=A, vq=A, vs=A, kv=A, B=2, Hkv=2, D=64, n_max=16, kc=A, vc=A, ws=A, wsb=256) | kw
        return fm.lib.fmlp_kv_read_q8(a["kq"], a["ks"], a["vq"], a["vs"], a["kv"], a["B"], a["Hkv"], a["D"], a["n_max"],
                                      a["kc"], a["vc"], a["ws"], a["wsb"], None)
    for bad in (dict(kq=None), dict(vq=MIS), dict(ks=None), dict(vs=MIS4), dict(kv=None), dict(B=0), dict(Hkv=0),
                dict(D=32), dict(n_max=0), dict(kc=MIS), dict(vc=None), dict(ws=None), dict(wsb=16)):
        assert read(**bad) == fm.FMLP_ERR_INVALID_ARG, bad


def tensors():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    return dict(q=bf(5, 4, 64), k=bf(5, 2, 64), v=bf(5, 2, 64), cu_seqlens=i32(4), kv_len=i32(3), rope=rope(),
                q_out=bf(5, 4, 64), k_cache=bf(3, 2, 16, 64), v_cache=bf(3, 2, 16, 64),
                workspace=torch.zeros(256, dtype=torch.uint8))


@pytest.mark.parametrize("bad,error", [
    (dict(q=torch.zeros(5, 4, 64)), TypeError), (dict(q=torch.zeros(5, 256, dtype=torch.bfloat16)), ValueError),
    (dict(k=torch.zeros(5, 3, 64, dtype=torch.bfloat16)), ValueError),
    (dict(v=torch.zeros(4, 2, 64, dtype=torch.bfloat16)), ValueError),
    (dict(q=torch.zeros(4, 5, 64, dtype=torch.bfloat16).transpose(0, 1)), ValueError),
    (dict(q=torch.zeros(1, 4, 64, dtype=torch.bfloat16).expand(5, 4, 64)), ValueError),
    (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(kv_len=torch.zeros(3, dtype=torch.int64)), TypeError), (dict(rope=1e4), TypeError),
    (dict(q_out=torch.zeros(5, 4, 64)), TypeError), (dict(k_cache=torch.zeros(3, 2, 16, 64)), TypeError),
    (dict(v_cache=torch.zeros(3, 2, 15, 64, dtype=torch.bfloat16)), ValueError),
    (dict(workspace=torch.zeros(255, dtype=torch.uint8)), ValueError),
    (dict(q_gamma=torch.zeros(65, dtype=torch.bfloat16)), ValueError),
    (dict(), ValueError),                                        # host tensors
])
def test_binding_checks(bad, error):
    with pytest.raises(error):
        fm.fmlp_rope_append(**(tensors() | bad))


def test_prefill_workspace_and_refusals():
    L = fm.lib
    assert L.fmlp_prefill_workspace_bytes(2048, 1, 32, 8, 128) >= 2 * 148 * 2 * 128 * 130 * 4
    assert L.fmlp_prefill_workspace_bytes(1, 1, 32, 8, 128) < L.fmlp_prefill_workspace_bytes(64, 1, 32, 8, 128)
    assert L.fmlp_prefill_workspace_bytes(0, 1, 8, 8, 64) > 0
    for T, B, H, Hkv, D in [(-1, 1, 8, 8, 64), (1, 0, 8, 8, 64), (1, 1, 12, 8, 64), (1, 1, 0, 1, 64), (1, 1, 8, 0, 64),
                            (1, 1, 8, 8, 80), (1 << 25, 1, 8, 8, 64), (1, 1, 258, 2, 64)]:
        assert L.fmlp_prefill_workspace_bytes(T, B, H, Hkv, D) == 0
    big = 1 << 30

    def attend(**kw):
        a = dict(q=A, qs=256, kc=A << 8, vc=A << 12, cu=A, kv=A, T=4, B=2, H=4, Hkv=2, D=64, n_max=16, scale=0.1,
                 out=0x900000, ws=A, wsb=big) | kw
        return L.fmlp_attn_prefill(a["q"], a["qs"], a["kc"], a["vc"], a["cu"], a["kv"], a["T"], a["B"], a["H"],
                                   a["Hkv"], a["D"], a["n_max"], a["scale"], a["out"], a["ws"], a["wsb"], None)
    assert attend(T=0, q=None, out=None) == fm.FMLP_OK
    for bad in (dict(q=None), dict(q=MIS), dict(qs=248), dict(qs=260), dict(kc=None), dict(vc=MIS), dict(cu=None),
                dict(kv=MIS4), dict(T=-1), dict(B=0), dict(H=3), dict(D=32), dict(n_max=0), dict(scale=0.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(out=MIS), dict(out=A + 16),
                dict(out=(A << 8) + 32), dict(out=A << 12), dict(ws=None), dict(ws=MIS), dict(wsb=1024),
                dict(B=65536, H=1024, Hkv=1024)):
        assert attend(**bad) == fm.FMLP_ERR_INVALID_ARG, bad


def test_prefill_binding_checks():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    good = dict(q=bf(5, 4, 64), k_cache=bf(3, 2, 16, 64), v_cache=bf(3, 2, 16, 64),
                cu_seqlens=torch.zeros(4, dtype=torch.int32), kv_len=torch.zeros(3, dtype=torch.int32), scale=0.1,
                out=bf(5, 4, 64), workspace=torch.zeros(1 << 24, dtype=torch.uint8))
    for bad, error in ((dict(q=torch.zeros(5, 4, 64)), TypeError), (dict(out=bf(5, 4, 65)), ValueError),
                       (dict(out=torch.zeros(5, 4, 64)), TypeError), (dict(k_cache=bf(3, 2, 64)), ValueError),
                       (dict(v_cache=bf(3, 2, 17, 64)), ValueError), (dict(kv_len=torch.zeros(2, dtype=torch.int32)), ValueError),
                       (dict(workspace=torch.zeros(64, dtype=torch.uint8)), ValueError),
                       (dict(q=bf(5, 3, 64), out=bf(5, 3, 64)), fm.FmlpError), (dict(), ValueError)):
        with pytest.raises(error):
            fm.fmlp_attn_prefill(**(good | bad))


def test_attn_q8_workspace_and_refusals():
    L = fm.lib
    assert L.fmlp_attn_q8_workspace_bytes(1, 32, 8, 128) >= 2 * 148 * 4 * 131 * 4
    for B, H, Hkv, D in [(0, 8, 8, 64), (1, 12, 8, 64), (1, 0, 1, 64), (1, 8, 8, 80), (1, 34, 2, 64), (70000, 8, 8, 64)]:
        assert L.fmlp_attn_q8_workspace_bytes(B, H, Hkv, D) == 0

    def attend(**kw):
        a = dict(q=A, kq=A, ks=A, vq=A, vs=A, kv=A, B=2, H=4, Hkv=2, D=64, n_max=16, scale=0.1, out=0x900000, ws=A,
                 wsb=1 << 30) | kw
        return L.fmlp_attn_decode_q8(a["q"], a["kq"], a["ks"], a["vq"], a["vs"], a["kv"], a["B"], a["H"], a["Hkv"],
                                     a["D"], a["n_max"], a["scale"], a["out"], a["ws"], a["wsb"], None)
    for bad in (dict(q=None), dict(q=MIS), dict(kq=None), dict(kq=MIS), dict(ks=None), dict(vs=MIS4), dict(vq=MIS),
                dict(kv=None), dict(kv=MIS4), dict(B=0), dict(H=3), dict(H=34), dict(D=32), dict(n_max=0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(out=None), dict(out=MIS), dict(out=A + 32),
                dict(kq=0x900000), dict(vs=0x900100), dict(ws=None), dict(wsb=300)):
        assert attend(**bad) == fm.FMLP_ERR_INVALID_ARG, bad
