"""Lengths that the packed-batch calls refuse, sequence by sequence: cu_seqlens that decrease or
leave [0, T] and kv_len outside [0, n_max] are reported, their sequences left as they were, and the
other sequences done.  Batches of up to 32, up to 256 and more sequences, whose tokens the append
finds in different ways."""

import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu

H, H_KV, D, N_MAX = 4, 2, 64, 32
ROPE = dict(theta=1e4, rotary_dim=64)


@pytest.fixture(scope="module")
def fm(cuda_device):
    import token_phase_swiglu_b200 as fm
    return fm


def setup(dev, cu, kv_len, T, seed):
    B = len(kv_len)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    return dict(q=wl.normal_bf16(seed, 70, (T, H, D)).to(dev), k=wl.normal_bf16(seed, 71, (T, H_KV, D)).to(dev),
                v=wl.normal_bf16(seed, 72, (T, H_KV, D)).to(dev), cu=i32(cu), kv_len=i32(kv_len),
                q_out=torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=dev),
                k_cache=torch.full((B, H_KV, N_MAX, D), 7.0, dtype=torch.bfloat16, device=dev),
                v_cache=torch.full((B, H_KV, N_MAX, D), 7.0, dtype=torch.bfloat16, device=dev),
                k_q=torch.full((B, H_KV, N_MAX, D), 7, dtype=torch.int8, device=dev),
                v_q=torch.full((B, H_KV, N_MAX, D), 7, dtype=torch.int8, device=dev),
                k_s=torch.full((B, H_KV, N_MAX), 7.0, device=dev), v_s=torch.full((B, H_KV, N_MAX), 7.0, device=dev),
                ws=torch.zeros(256, dtype=torch.uint8, device=dev))


def append(fm, s, q8):
    head = (s["q"], s["k"], s["v"], s["cu"], s["kv_len"], fm.FmlpRope(**ROPE), s["q_out"])
    if q8:
        fm.fmlp_rope_append_q8(*head, s["k_q"], s["k_s"], s["v_q"], s["v_s"], s["ws"])
    else:
        fm.fmlp_rope_append(*head, s["k_cache"], s["v_cache"], s["ws"])
    return fm.fmlp_device_status(s["ws"])


# cu, kv_len (of the first sequences; the batch is filled up with sequences of no tokens), T, refused
BATCHES = [
    ([0, 20], [25], 10, {0}),                               # leaves [0, T]
    ([0, 3, 8, 13], [9, 20, 30], 12, {2}),
    ([-3, 4, 9], [9, 20], 12, {0}),                         # starts before the first token
    ([0, 5, 3], [9, 9], 8, {1}),                            # decreases at the end
    ([4, 2, 6], [9, 9], 8, {0}),                            # decreases at the start
    ([0, 4, 2, 2], [9, 9, 9], 8, {1}),
    ([0, 3, 3, 6], [9, N_MAX + 1, 9], 8, {1}),              # a bad length of a sequence without tokens
    ([0, 3, 3, 6], [9, -1, 9], 8, {1}),
    ([0, 3, 5, 6], [9, -2000000000, 9], 8, {1}),
    ([0, 2147483647, 6], [9, 9], 8, {0, 1}),
    ([-2147483648, 2, 6], [9, 9], 8, {0}),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B", [0, 32, 33, 256, 700])
@pytest.mark.parametrize("cu,kv_len,T,bad", BATCHES)
def test_append_refuses_a_sequence_and_does_the_others(fm, cuda_device, cu, kv_len, T, bad, B, q8):
    # sequences without tokens: in front of the others, or (in range only) behind them
    fill = max(0, B - len(kv_len))
    front = fill // 2 if 0 <= cu[0] <= T else 0
    behind = fill - front if 0 <= cu[-1] <= T else 0
    cu = [cu[0]] * front + cu + [cu[-1]] * behind
    kv_len = [0] * front + kv_len + [N_MAX] * behind
    bad = {b + front for b in bad}
    s = setup(cuda_device, cu, kv_len, T, seed=len(cu))
    assert append(fm, s, q8) == fm.FMLP_ERR_INVALID_ARG
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK          # reading clears it
    # each well-formed sequence as in a batch of its own
    want = setup(cuda_device, cu, kv_len, T, seed=len(cu))
    for b in range(len(kv_len)):
        if b in bad or cu[b] == cu[b + 1]:
            continue
        one = setup(cuda_device, [cu[b], cu[b + 1]], [kv_len[b]], T, seed=len(cu))
        assert append(fm, one, q8) == fm.FMLP_OK
        want["q_out"][cu[b]:cu[b + 1]] = one["q_out"][cu[b]:cu[b + 1]]
        for c in ("k_cache", "v_cache", "k_q", "v_q", "k_s", "v_s"):
            want[c][b] = one[c][0]
    for c in ("q_out", "k_cache", "v_cache", "k_q", "v_q", "k_s", "v_s"):
        assert torch.equal(s[c], want[c]), c


@pytest.mark.parametrize("B", [1, 31, 32, 33, 256, 257, 2000])
def test_padded_batches_are_not_reported(fm, cuda_device, B):
    """Tokens of no sequence in front and behind, sequences without tokens and tokens without rows."""
    n = [(b * 5) % 3 for b in range(B)]
    cu = [4]
    for x in n:
        cu.append(cu[-1] + x)
    kv_len = [(b * 7) % 4 for b in range(B)]
    T = cu[-1] + 6
    s = setup(cuda_device, cu, kv_len, T, seed=B)
    assert append(fm, s, False) == fm.FMLP_OK
    row = [None] * T
    for b in range(B):
        for i in range(n[b]):
            if kv_len[b] - n[b] + i >= 0:
                row[cu[b] + i] = (b, kv_len[b] - n[b] + i)
    want = torch.full_like(s["v_cache"], 7.0)
    for t, at in enumerate(row):
        if at is not None:
            want[at[0], :, at[1]] = s["v"][t]
    written = torch.tensor([at is not None for at in row], device=cuda_device)
    assert torch.equal(s["v_cache"], want)
    assert torch.all(s["q_out"][~written] == 7) and not torch.any((s["q_out"][written] == 7).all(-1))


def test_attention_refuses_the_same_batches(fm, cuda_device):
    for cu, kv_len, T, bad in BATCHES:
        s = setup(cuda_device, cu, kv_len, T, seed=3)
        B = len(kv_len)
        ws = torch.zeros(fm.fmlp_prefill_workspace_bytes(T, B, H, H_KV, D), dtype=torch.uint8, device=cuda_device)
        s["k_cache"].normal_()
        s["v_cache"].normal_()
        fm.fmlp_attn_prefill(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["kv_len"], 0.125, s["q_out"], ws)
        assert fm.fmlp_device_status(ws) == fm.FMLP_ERR_INVALID_ARG
        done = torch.zeros(T, dtype=torch.bool, device=cuda_device)
        for b in range(B):
            if b not in bad:
                done[cu[b]:cu[b + 1]] = True
        assert torch.all(s["q_out"][~done] == 7) and not torch.any((s["q_out"][done] == 7).all(-1))
