"""Memory that a packed-batch call may not share between what it writes and what it reads, or between
two things it writes: refused on the host, byte-exact at both ends; what touches without
overlapping, and what is only read twice, is taken.  Addresses are made up, so nothing here may reach a GPU."""

import ctypes

import pytest
import torch

import token_phase_swiglu_b200 as fm

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")

T, B, H, HKV, D, N = 5, 3, 4, 2, 64, 16
L = fm.lib
Q_ROW, KV_ROW, ROWS = H * D, HKV * D, B * HKV * N
STRIDE = Q_ROW + 2 * KV_ROW + 8

# name -> (bytes, written)
APPEND = dict(q=(((T - 1) * STRIDE + Q_ROW) * 2, False), k=(((T - 1) * STRIDE + KV_ROW) * 2, False),
              v=(((T - 1) * STRIDE + KV_ROW) * 2, False), cu=((B + 1) * 4, False), kv=(B * 4, False),
              qg=(D * 2, False), kg=(D * 2, False), qo=(T * Q_ROW * 2, True), kc=(ROWS * D * 2, True),
              vc=(ROWS * D * 2, True), ws=(256, True))
APPEND_Q8 = APPEND | dict(kc=(ROWS * D, True), vc=(ROWS * D, True), ks=(ROWS * 4, True), vs=(ROWS * 4, True))
READ = dict(kq=(ROWS * D, False), vq=(ROWS * D, False), ks=(ROWS * 4, False), vs=(ROWS * 4, False), kv=(B * 4, False),
            kc=(ROWS * D * 2, True), vc=(ROWS * D * 2, True), ws=(256, True))
PREFILL = dict(q=(((T - 1) * STRIDE + Q_ROW) * 2, False), kc=(ROWS * D * 2, False), vc=(ROWS * D * 2, False),
               cu=((B + 1) * 4, False), kv=(B * 4, False), out=(T * Q_ROW * 2, True),
               ws=(L.fmlp_prefill_workspace_bytes(T, B, H, HKV, D), True))
DECODE = dict(q=(B * Q_ROW * 2, False), kq=(ROWS * D, False), vq=(ROWS * D, False), ks=(ROWS * 4, False),
              vs=(ROWS * 4, False), kv=(B * 4, False), out=(B * Q_ROW * 4, True),
              ws=(L.fmlp_attn_q8_workspace_bytes(B, H, HKV, D), True))


def place(parts):
    """An address for each, 16 MB apart (more than any of them takes)."""
    return {name: (i + 1) << 24 for i, name in enumerate(parts)}


def append(a, q_stride=STRIDE, n_max=N, b=B):
    r = fm.FmlpRope(1e4, D)
    pre = [a["q"], q_stride, a["k"], STRIDE, a["v"], STRIDE, T, a["cu"], a["kv"], b, H, HKV, D, ctypes.byref(r._c),
           a["qg"], a["kg"], 1e-6, a["qo"]]
    if "ks" in a:
        return L.fmlp_rope_append_q8(*pre, a["kc"], a["ks"], a["vc"], a["vs"], n_max, a["ws"], 256, None)
    return L.fmlp_rope_append(*pre, a["kc"], a["vc"], n_max, a["ws"], 256, None)


def read(a):
    return L.fmlp_kv_read_q8(a["kq"], a["ks"], a["vq"], a["vs"], a["kv"], B, HKV, D, N, a["kc"], a["vc"], a["ws"], 256, None)


def prefill(a):
    return L.fmlp_attn_prefill(a["q"], STRIDE, a["kc"], a["vc"], a["cu"], a["kv"], T, B, H, HKV, D, N, 0.1, a["out"],
                               a["ws"], PREFILL["ws"][0], None)


def decode(a):
    return L.fmlp_attn_decode_q8(a["q"], a["kq"], a["ks"], a["vq"], a["vs"], a["kv"], B, H, HKV, D, N, 0.1, a["out"],
                                 a["ws"], DECODE["ws"][0], None)


CALLS = [(append, APPEND), (append, APPEND_Q8), (read, READ), (prefill, PREFILL), (decode, DECODE)]


def test_apart_is_taken():
    for call, parts in CALLS:
        assert call(place(parts)) not in (fm.FMLP_OK, fm.FMLP_ERR_INVALID_ARG)


@pytest.mark.parametrize("call,parts", CALLS, ids=["append", "append_q8", "read_q8", "prefill", "decode_q8"])
def test_every_pair(call, parts):
    for x, (size, written) in parts.items():
        for y, (other, written_too) in parts.items():
            if x == y:
                continue
            base = place(parts)
            end = base[x] + size                                   # y begins at the last 16 bytes of x, or behind x
            inside, behind = (end - 1) // 16 * 16, (end + 15) // 16 * 16
            refused = written or written_too
            assert (call(base | {y: inside}) == fm.FMLP_ERR_INVALID_ARG) == refused, (x, y)
            assert (call(base | {y: base[x]}) == fm.FMLP_ERR_INVALID_ARG) == refused, (x, y)
            assert call(base | {y: behind}) != fm.FMLP_ERR_INVALID_ARG, (x, y)


def test_in_place_queries():
    for parts in (APPEND, APPEND_Q8):
        base = place(parts)
        base["qo"] = base["q"]
        assert append(base, q_stride=Q_ROW) != fm.FMLP_ERR_INVALID_ARG
        assert append(base) == fm.FMLP_ERR_INVALID_ARG             # rows of the output would fall between the input's
        assert append(base | {"k": base["q"]}, q_stride=Q_ROW) == fm.FMLP_ERR_INVALID_ARG


def test_without_norms():
    base = place(APPEND) | {"qg": None, "kg": None}
    assert append(base) not in (fm.FMLP_OK, fm.FMLP_ERR_INVALID_ARG)


def test_caches_larger_than_any_memory():
    """Their size does not wrap round to a small one."""
    base = place(APPEND)
    r = fm.FmlpRope(1e4, 128)
    a = base
    args = [a["q"], 1 << 17, a["k"], 1 << 17, a["v"], 1 << 17, T, a["cu"], a["kv"], 65536, 1024, 1024, 128, ctypes.byref(r._c),
            None, None, 1e-6, a["qo"], a["kc"], a["vc"], (1 << 30) - 1, a["ws"], 256, None]
    assert L.fmlp_rope_append(*args) == fm.FMLP_ERR_INVALID_ARG
