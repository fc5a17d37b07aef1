"""The packed-batch calls run together, as a serving loop runs them: a ragged batch of
prompts is rotated, appended and attended, decode steps follow on the same cache (by
fmlp_attn_decode, which rotates and appends on its own, and by the packed calls with one
token a sequence), and the same batch goes through an int8 cache.

The bf16 path is compared step by step with the oracle fed the caches as the GPU holds
them (their contents are checked where they are written), at the tolerance of each call:
2^-8 (|o| + A) + 2^-11 A for fmlp_attn_prefill (see test_prefill.py) and normwise 1e-4 for
fmlp_attn_decode (see test_attn.py)."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import decode_bf16, packed
import workloads as wl

pytestmark = pytest.mark.gpu

B, H, H_KV, D, N_MAX, THETA = 3, 8, 2, 128, 300, 10000.0
PROMPTS = [200, 37, 129]


@pytest.fixture(scope="module")
def fm(cuda_device):
    import token_phase_swiglu_b200 as fm
    return fm


def dec(t):
    return decode_bf16(wl.bf16_bits(t.detach().cpu()))


def i32(dev, x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def qkv(dev, T, seed):
    x = wl.normal_bf16(seed, 70, (T, (H + 2 * H_KV) * D)).to(dev)
    q, k, v = x.split((H * D, H_KV * D, H_KV * D), dim=1)
    return q.unflatten(1, (H, D)), k.unflatten(1, (H_KV, D)), v.unflatten(1, (H_KV, D))


def check_prefill(out, q_rot, k_cache, v_cache, cu, lens, scale):
    q, k, v = dec(q_rot), dec(k_cache), dec(v_cache)
    o = packed.causal_attention(q, k, v, cu, lens, scale)
    a = packed.causal_attention(q, k, np.abs(v), cu, lens, scale)
    assert np.all(np.abs(dec(out) - o) <= 2.0 ** -8 * (np.abs(o) + a) + 2.0 ** -11 * a)


def test_prompts_then_decode_steps(fm, cuda_device):
    dev, rope, scale = cuda_device, fm.FmlpRope(THETA, D), 1 / math.sqrt(D)
    k_cache = torch.zeros(B, H_KV, N_MAX, D, dtype=torch.bfloat16, device=dev)
    v_cache = torch.zeros_like(k_cache)
    T, cu = sum(PROMPTS), [0, *np.cumsum(PROMPTS).tolist()]
    ws = torch.zeros(max(fm.fmlp_prefill_workspace_bytes(T, B, H, H_KV, D),
                         fm.fmlp_attn_workspace_bytes(B, H, H_KV, D)), dtype=torch.uint8, device=dev)
    q, k, v = qkv(dev, T, 1)
    q_rot, out = (torch.empty(T, H, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    fm.fmlp_rope_append(q, k, v, i32(dev, cu), i32(dev, PROMPTS), rope, q_rot, k_cache, v_cache, ws)
    fm.fmlp_attn_prefill(q_rot, k_cache, v_cache, i32(dev, cu), i32(dev, PROMPTS), scale, out, ws)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    check_prefill(out, q_rot, k_cache, v_cache, cu, PROMPTS, scale)
    # the token-phase step goes on from the prompts' cache
    q, k, v = (t.contiguous() for t in qkv(dev, B, 2))
    before = dec(k_cache), dec(v_cache)
    step = torch.empty(B, H, D, device=dev)
    ws.zero_()
    fm.fmlp_attn_decode(q, k, v, k_cache, v_cache, i32(dev, PROMPTS), max(PROMPTS) + 1, THETA, step, ws)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    ref, _, _ = oracle.token_attention(dec(q), dec(k), dec(v), *before, np.array(PROMPTS), THETA)
    got = step.cpu().double().numpy()
    assert np.linalg.norm(got - ref) / np.linalg.norm(ref) <= 1e-4
    # and so do the packed calls, with 1, 3 and no new tokens
    new, lens = [1, 3, 0], [PROMPTS[0] + 2, PROMPTS[1] + 4, PROMPTS[2] + 1]
    cu = [0, 1, 4, 4]
    ws.zero_()
    q, k, v = qkv(dev, sum(new), 3)
    q_rot, out = (torch.empty(sum(new), H, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    fm.fmlp_rope_append(q, k, v, i32(dev, cu), i32(dev, lens), rope, q_rot, k_cache, v_cache, ws)
    fm.fmlp_attn_prefill(q_rot, k_cache, v_cache, i32(dev, cu), i32(dev, lens), scale, out, ws)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    check_prefill(out, q_rot, k_cache, v_cache, cu, lens, scale)


def test_one_token_agrees_with_the_token_phase_step(fm, cuda_device):
    """A decode step by fmlp_attn_decode and by fmlp_rope_append + fmlp_attn_prefill write the same
    cache rows (to a bf16 step) and give the same result to bf16."""
    dev, pos = cuda_device, [250, 0, 63]
    p = wl.make_attn_problem(B, H, H_KV, D, N_MAX, seed=4)
    g = {key: t.to(dev) for key, t in p.items()}
    caches = [(g["k_cache"].clone(), g["v_cache"].clone()) for _ in range(2)]
    ws = torch.zeros(fm.fmlp_attn_workspace_bytes(B, H, H_KV, D), dtype=torch.uint8, device=dev)
    one = torch.empty(B, H, D, device=dev)
    fm.fmlp_attn_decode(g["q"], g["k_new"], g["v_new"], *caches[0], i32(dev, pos), max(pos) + 1, THETA, one, ws)
    cu, lens = i32(dev, [0, 1, 2, 3]), i32(dev, [x + 1 for x in pos])
    ws2 = torch.zeros(fm.fmlp_prefill_workspace_bytes(B, B, H, H_KV, D), dtype=torch.uint8, device=dev)
    q_rot, two = (torch.empty(B, H, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    fm.fmlp_rope_append(g["q"], g["k_new"], g["v_new"], cu, lens, fm.FmlpRope(THETA, D), q_rot, *caches[1], ws2)
    fm.fmlp_attn_prefill(q_rot, *caches[1], cu, lens, 1 / math.sqrt(D), two, ws2)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK and fm.fmlp_device_status(ws2) == fm.FMLP_OK
    assert torch.equal(caches[0][1], caches[1][1])
    a, b = caches[0][0].float(), caches[1][0].float()
    assert torch.all((a - b).abs() <= 2.0 ** -7 * b.abs())
    # q rotated to bf16 moves a score by 2^-8 of |q||k| scale at most, some 1e-2: weights by 1%
    assert torch.all((one - two.float()).abs() <= 0.03 * one.abs().amax(-1, keepdim=True) + 0.03)


def test_int8_cache_from_prompt_to_decode_captured(fm, cuda_device):
    """Prompts into an int8 cache and read back for their attention, then a decode step captured once
    and replayed with growing lengths."""
    dev, rope, scale = cuda_device, fm.FmlpRope(THETA, D), 1 / math.sqrt(D)
    kq, vq = (torch.zeros(B, H_KV, N_MAX, D, dtype=torch.int8, device=dev) for _ in range(2))
    ks, vs = (torch.zeros(B, H_KV, N_MAX, device=dev) for _ in range(2))
    k16, v16 = (torch.zeros(B, H_KV, N_MAX, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    T, cu = sum(PROMPTS), [0, *np.cumsum(PROMPTS).tolist()]
    ws = torch.zeros(max(fm.fmlp_prefill_workspace_bytes(T, B, H, H_KV, D),
                         fm.fmlp_attn_q8_workspace_bytes(B, H, H_KV, D)), dtype=torch.uint8, device=dev)
    q, k, v = qkv(dev, T, 5)
    q_rot, out = (torch.empty(T, H, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    fm.fmlp_rope_append_q8(q, k, v, i32(dev, cu), i32(dev, PROMPTS), rope, q_rot, kq, ks, vq, vs, ws)
    fm.fmlp_kv_read_q8(kq, ks, vq, vs, i32(dev, PROMPTS), k16, v16, ws)
    fm.fmlp_attn_prefill(q_rot, k16, v16, i32(dev, cu), i32(dev, PROMPTS), scale, out, ws)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    check_prefill(out, q_rot, k16, v16, cu, PROMPTS, scale)
    # decode: append and attend, captured
    q, k, v = qkv(dev, B, 6)
    one, lens = i32(dev, [0, 1, 2, 3]), i32(dev, [n + 1 for n in PROMPTS])
    q1, o1 = torch.empty(B, H, D, dtype=torch.bfloat16, device=dev), torch.empty(B, H, D, device=dev)

    def step():
        fm.fmlp_rope_append_q8(q, k, v, one, lens, rope, q1, kq, ks, vq, vs, ws)
        fm.fmlp_attn_decode_q8(q1, kq, ks, vq, vs, lens, scale, o1, ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for more in (1, 2, 3):
        lens.copy_(torch.tensor([n + more for n in PROMPTS]))
        g.replay()
        torch.cuda.synchronize()
        assert fm.fmlp_device_status(ws) == fm.FMLP_OK
        ref = packed.decode_attention_q8(dec(q1), kq.cpu().numpy(), ks.cpu().numpy(), vq.cpu().numpy(),
                                         vs.cpu().numpy(), lens.cpu().numpy(), scale)
        got = o1.cpu().double().numpy()
        assert np.linalg.norm(got - ref) / np.linalg.norm(ref) <= 1e-5


def test_two_streams_with_their_own_workspaces(fm, cuda_device):
    """Two batches at once on two streams, each with its workspace."""
    dev, scale = cuda_device, 1 / math.sqrt(D)
    work = []
    for seed in (7, 8):
        p = wl.make_attn_problem(B, H, H_KV, D, N_MAX, seed=seed)
        s = dict(k=p["k_cache"].to(dev), v=p["v_cache"].to(dev), q=wl.normal_bf16(seed, 71, (60, H, D)).to(dev),
                 out=torch.zeros(60, H, D, dtype=torch.bfloat16, device=dev), cu=i32(dev, [0, 20, 21, 60]),
                 lens=i32(dev, [300, 77, 200]), st=torch.cuda.Stream(),
                 ws=torch.zeros(fm.fmlp_prefill_workspace_bytes(60, B, H, H_KV, D), dtype=torch.uint8, device=dev))
        work.append(s)
    torch.cuda.synchronize()
    for _ in range(5):
        for s in work:
            fm.fmlp_attn_prefill(s["q"], s["k"], s["v"], s["cu"], s["lens"], scale, s["out"], s["ws"], stream=s["st"])
    torch.cuda.synchronize()
    for s in work:
        assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
        check_prefill(s["out"], s["q"], s["k"], s["v"], [0, 20, 21, 60], [300, 77, 200], scale)


def test_one_workspace_for_all_calls_in_any_order(fm, cuda_device):
    """Prompt attention and int8 decode attention, both split over many CTAs, take turns on one
    workspace: each finds its counters as it needs them."""
    dev, scale, n = cuda_device, 1 / math.sqrt(D), 6000
    ws = torch.zeros(max(fm.fmlp_prefill_workspace_bytes(150, 1, H, H_KV, D),
                         fm.fmlp_attn_q8_workspace_bytes(1, H, H_KV, D)), dtype=torch.uint8, device=dev)
    kc, vc = (wl.normal_bf16(9, i, (1, H_KV, n, D)).to(dev) for i in (72, 73))
    kq, vq = (torch.randint(-127, 128, (1, H_KV, n, D), dtype=torch.int8, device=dev) for _ in range(2))
    ks, vs = (torch.rand(1, H_KV, n, device=dev) / 64 for _ in range(2))
    q = wl.normal_bf16(9, 74, (150, H, D)).to(dev)
    cu, lens = i32(dev, [0, 150]), i32(dev, [n])
    out, one = torch.empty(150, H, D, dtype=torch.bfloat16, device=dev), torch.empty(1, H, D, device=dev)
    seen = []
    for _ in range(4):
        fm.fmlp_attn_prefill(q, kc, vc, cu, lens, scale, out, ws)
        fm.fmlp_attn_decode_q8(q[:1], kq, ks, vq, vs, lens, scale, one, ws)
        assert fm.fmlp_device_status(ws) == fm.FMLP_OK
        seen.append((out.clone(), one.clone()))
        out.zero_(), one.zero_()
    assert all(torch.equal(a, seen[0][0]) and torch.equal(b, seen[0][1]) for a, b in seen)
    ref = packed.decode_attention_q8(dec(q[:1]), kq.cpu().numpy(), ks.cpu().numpy(), vq.cpu().numpy(),
                                     vs.cpu().numpy(), [n], scale)
    assert np.linalg.norm(seen[0][1].cpu().double().numpy() - ref) / np.linalg.norm(ref) <= 1e-5
    z = torch.softmax(q[149, 0].double() @ kc[0, 0].double().T * scale, -1)
    want, a = z @ vc[0, 0].double(), z @ vc[0, 0].double().abs()
    got = seen[0][0][149, 0].double()
    assert torch.all((got - want).abs() <= 2.0 ** -8 * (want.abs() + a) + 2.0 ** -11 * a)
