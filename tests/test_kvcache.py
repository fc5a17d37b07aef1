"""fmlp_rope_append, fmlp_rope_append_q8 and fmlp_kv_read_q8 against the binary64 oracle.

Tolerances.  A bf16 output is the f32 result rounded once: half a step, 2^-8 of
the value.  The f32 result itself: with x, the cosine and the sine each off by
at most 2^-24 relative (the norm's product adds a handful of such roundings),
|y - y_ref| <= 16 * 2^-24 (|x0| + |x1|) * amplitude, so every element is asked
to be within 2^-8 |y| + 2^-20 (|x0| + |x1|) amplitude.  Values in a bf16 cache
are copied and have to be equal.
The int8 cache: with an f32 result off by e, the scale is off by at most
e/127 + 2^-24 s, and a code may step over where x / s sits next to a half; what
a row stands for is then off by half a scale step (its rounding) plus e and the
scale's error: (0.5 + 2^-10) s for every element.  Codes differ from the oracle's
by at most 1, and rarely."""

import numpy as np
import pytest
import torch

from oracle import decode_bf16, packed
import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm(cuda_device):
    import token_phase_swiglu_b200 as fm
    return fm


def dec(t):
    return decode_bf16(wl.bf16_bits(t.detach().cpu()))


def batch(dev, lens, H, H_kv, D, n_max, seed, front=0, behind=0):
    """A packed batch as column ranges of one tensor; `front`/`behind`: tokens of no sequence."""
    cu = [front]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    T = cu[-1] + behind
    qkv = wl.normal_bf16(seed, 40, (T, (H + 2 * H_kv) * D)).to(dev)
    q, k, v = qkv.split((H * D, H_kv * D, H_kv * D), dim=1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    return dict(q=q.unflatten(1, (H, D)), k=k.unflatten(1, (H_kv, D)), v=v.unflatten(1, (H_kv, D)), cu=i32(cu),
                kv_len=i32([x for _, x in lens]), cu_list=cu, len_list=[x for _, x in lens], T=T,
                qg=wl.normal_bf16(seed, 41, (D,), mean=1.0, std=0.2).to(dev),
                kg=wl.normal_bf16(seed, 42, (D,), mean=1.0, std=0.2).to(dev),
                ws=torch.zeros(256, dtype=torch.uint8, device=dev),
                k_cache=wl.normal_bf16(seed, 43, (len(lens), H_kv, n_max, D)).to(dev),
                v_cache=wl.normal_bf16(seed, 44, (len(lens), H_kv, n_max, D)).to(dev),
                q_out=torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=dev))


def reference(s, rot, norms, which, eps=1e-6):
    """(values, bound on the f32 error) of q or k, per token; None where nothing is written."""
    x = dec(s[which].contiguous())
    gamma = dec(s[which + "g"]) if norms else None
    freq = packed.rope_frequencies(rot["theta"], rot["rotary_dim"],
                                   **{k: rot[k] for k in ("scaling", "factor", "low", "high", "original_ctx") if k in rot})
    amp, R, inter = rot.get("amplitude", 1.0), rot["rotary_dim"], rot.get("interleaved", False)
    out = []
    for t, at in enumerate(packed.positions(s["cu_list"], s["len_list"], s["T"])):
        if at is None:
            out.append(None)
            continue
        y = packed.head_norm(x[t], gamma, eps) if norms else x[t]
        a = np.abs(y)
        size = a.copy()
        if R:
            lo = np.arange(0, R, 2) if inter else np.arange(R // 2)
            hi = lo + 1 if inter else lo + R // 2
            size[:, lo] = size[:, hi] = (a[:, lo] + a[:, hi]) * max(1.0, amp)
        out.append((packed.rotate(y, at[1], freq, inter, amp), 2.0 ** -20 * size))
    return out


CASES = [
    # lens (new, held), H, H_kv, D, n_max, rotation, norms
    ([(1, 1)], 4, 2, 64, 8, dict(theta=1e4, rotary_dim=64), False),
    ([(3, 5), (0, 4), (1, 16), (17, 17)], 8, 1, 128, 17, dict(theta=5e5, rotary_dim=128), True),
    ([(5, 9), (2, 2)], 6, 2, 96, 9, dict(theta=1e4, rotary_dim=48, interleaved=True, scaling="linear", factor=4.0), True),
    ([(33, 40)], 1, 1, 96, 41, dict(theta=1e4, rotary_dim=96, interleaved=True), False),
    ([(1, 599)] * 40, 32, 8, 128, 600,
     dict(theta=5e5, rotary_dim=128, scaling="bands", factor=8.0, low=1.0, high=4.0, original_ctx=128), False),
    ([(300, 300)], 3, 3, 64, 333,
     dict(theta=1e4, rotary_dim=32, scaling="yarn", factor=16.0, low=1.0, high=32.0, original_ctx=64, amplitude=1.2),
     True),
    ([(2, 70000)], 2, 1, 64, 70000, dict(theta=1e4, rotary_dim=0), True),
    ([(7, 100000)], 5, 1, 128, 100001, dict(theta=1e7, rotary_dim=16), False),
    # padding: more new tokens than rows, and none held
    ([(4, 2), (3, 0), (2, 2)], 4, 2, 64, 8, dict(theta=1e4, rotary_dim=64), False),
]


@pytest.mark.parametrize("lens,H,H_kv,D,n_max,rot,norms", CASES)
def test_append_matches_oracle(fm, cuda_device, lens, H, H_kv, D, n_max, rot, norms):
    s = batch(cuda_device, lens, H, H_kv, D, n_max, seed=len(lens) * 31 + D, front=2, behind=3)
    k0, v0 = s["k_cache"].clone(), s["v_cache"].clone()
    fm.fmlp_rope_append(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], fm.FmlpRope(**rot), s["q_out"], s["k_cache"],
                        s["v_cache"], s["ws"], q_gamma=s["qg"] if norms else None, k_gamma=s["kg"] if norms else None)
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    q_out = dec(s["q_out"])
    for t, r in enumerate(reference(s, rot, norms, "q")):
        if r is None:
            assert np.all(q_out[t] == 7.0)
        else:
            assert np.all(np.abs(q_out[t] - r[0]) <= 2.0 ** -8 * np.abs(r[0]) + r[1])
    at = packed.positions(s["cu_list"], s["len_list"], s["T"])
    for t, r in enumerate(reference(s, rot, norms, "k")):
        if r is None:
            continue
        b, p = at[t]
        got = dec(s["k_cache"][b, :, p])
        assert np.all(np.abs(got - r[0]) <= 2.0 ** -8 * np.abs(r[0]) + r[1])
        assert torch.equal(s["v_cache"][b, :, p], s["v"][t])
        k0[b, :, p], v0[b, :, p] = s["k_cache"][b, :, p], s["v_cache"][b, :, p]
    assert torch.equal(s["k_cache"], k0) and torch.equal(s["v_cache"], v0)   # no other row


@pytest.mark.parametrize("lens,H,H_kv,D,n_max,rot,norms", CASES)
def test_append_q8_and_read_back(fm, cuda_device, lens, H, H_kv, D, n_max, rot, norms):
    s = batch(cuda_device, lens, H, H_kv, D, n_max, seed=len(lens) * 37 + D, front=1)
    if s["T"] > 2:
        s["v"][-1, 0] = 0                                  # a row of zeros
    B = len(lens)
    codes = {c: torch.randint(-127, 128, (B, H_kv, n_max, D), dtype=torch.int8, device=cuda_device) for c in "kv"}
    scales = {c: torch.rand(B, H_kv, n_max, device=cuda_device) for c in "kv"}
    codes0, scales0 = {c: x.clone() for c, x in codes.items()}, {c: x.clone() for c, x in scales.items()}
    fm.fmlp_rope_append_q8(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], fm.FmlpRope(**rot), s["q_out"], codes["k"],
                           scales["k"], codes["v"], scales["v"], s["ws"], q_gamma=s["qg"] if norms else None,
                           k_gamma=s["kg"] if norms else None)
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    at = packed.positions(s["cu_list"], s["len_list"], s["T"])
    steps = total = 0
    rows = {"k": reference(s, rot, norms, "k"), "v": [(x, 0) for x in dec(s["v"].contiguous())]}
    for c in "kv":
        for t, where in enumerate(at):
            if where is None:
                continue
            b, p = where
            x = rows[c][t][0]
            ref_q, ref_s = packed.quantize_kv(x)
            q, sc = codes[c][b, :, p].cpu().numpy().astype(int), scales[c][b, :, p].cpu().double().numpy()
            assert np.all(np.abs(sc - ref_s) <= 2.0 ** -18 * ref_s)
            assert np.all(np.abs(q) <= 127) and np.all(np.abs(q - ref_q) <= 1)
            assert np.all(np.abs(q * sc[:, None] - x) <= (0.5 + 2.0 ** -10) * sc[:, None])
            steps, total = steps + np.sum(q != ref_q), total + q.size
            codes0[c][b, :, p], scales0[c][b, :, p] = codes[c][b, :, p], scales[c][b, :, p]
    assert steps <= max(2, 1e-3 * total)
    for c in "kv":
        assert torch.equal(codes[c], codes0[c]) and torch.equal(scales[c], scales0[c])
    # read back: code * scale rounded to bf16 once, rows behind kv_len untouched
    k0, v0 = s["k_cache"].clone(), s["v_cache"].clone()
    fm.fmlp_kv_read_q8(codes["k"], scales["k"], codes["v"], scales["v"], s["kv_len"], s["k_cache"], s["v_cache"],
                       s["ws"])
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    for b, n in enumerate(s["len_list"]):
        for c, old in (("k", k0), ("v", v0)):
            new = s[c + "_cache"]
            want = (codes[c][b, :, :n].float() * scales[c][b, :, :n, None]).to(torch.bfloat16)
            assert torch.equal(new[b, :, :n], want) and torch.equal(new[b, :, n:], old[b, :, n:])


def test_append_in_place_and_contiguous_rows(fm, cuda_device):
    lens, rot = [(9, 9), (20, 31)], dict(theta=1e4, rotary_dim=96)
    s = batch(cuda_device, lens, 4, 2, 96, 40, seed=3)
    q, k, v = (s[c].contiguous() for c in "qkv")
    args = (s["cu"], s["kv_len"], fm.FmlpRope(**rot))
    fm.fmlp_rope_append(s["q"], s["k"], s["v"], *args, s["q_out"], s["k_cache"], s["v_cache"], s["ws"],
                        q_gamma=s["qg"], k_gamma=s["kg"])
    k1, v1 = torch.zeros_like(s["k_cache"]), torch.zeros_like(s["v_cache"])
    fm.fmlp_rope_append(q, k, v, *args, q, k1, v1, s["ws"], q_gamma=s["qg"], k_gamma=s["kg"])
    assert torch.equal(q, s["q_out"])
    for b, (n, held) in enumerate(lens):
        assert torch.equal(k1[b, :, held - n:held], s["k_cache"][b, :, held - n:held])


def test_one_gamma_only(fm, cuda_device):
    s = batch(cuda_device, [(6, 6)], 4, 2, 64, 6, seed=4)
    rot = dict(theta=1e4, rotary_dim=64)
    fm.fmlp_rope_append(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], fm.FmlpRope(**rot), s["q_out"], s["k_cache"],
                        s["v_cache"], s["ws"], k_gamma=s["kg"])
    for which, norms, got in (("q", False, dec(s["q_out"])), ("k", True, dec(s["k_cache"])[0].transpose(1, 0, 2))):
        for t, r in enumerate(reference(s, rot, norms, which)):
            assert np.all(np.abs(got[t] - r[0]) <= 2.0 ** -8 * np.abs(r[0]) + r[1])


def test_bad_lengths_are_reported_and_skipped(fm, cuda_device):
    """A length past n_max, a negative one: the sequence is left as it was, the others are done."""
    s = batch(cuda_device, [(2, 2), (3, 99), (2, -1), (1, 8)], 2, 1, 64, 8, seed=5)
    k0 = s["k_cache"].clone()
    rope = fm.FmlpRope(1e4, 64)
    fm.fmlp_rope_append(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], rope, s["q_out"], s["k_cache"], s["v_cache"],
                        s["ws"])
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_ERR_INVALID_ARG
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK          # reading clears it
    assert torch.equal(s["k_cache"][1:3], k0[1:3]) and torch.all(s["q_out"][2:7] == 7)
    assert not torch.equal(s["k_cache"][0, :, :2], k0[0, :, :2]) and not torch.any(s["q_out"][7] == 7)
    # decreasing cu_seqlens
    s["cu"].copy_(torch.tensor([0, 5, 3, 7, 8]))
    s["kv_len"].copy_(torch.tensor([8, 8, 8, 8]))
    fm.fmlp_rope_append(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], rope, s["q_out"], s["k_cache"], s["v_cache"],
                        s["ws"])
    fm.fmlp_device_status(s["ws"])
    # read back: the bad sequence's rows stay
    codes = torch.ones(4, 1, 8, 64, dtype=torch.int8, device=cuda_device)
    scales = torch.ones(4, 1, 8, device=cuda_device)
    s["kv_len"].copy_(torch.tensor([1, 9, -5, 8]))
    k0 = s["k_cache"].clone()
    fm.fmlp_kv_read_q8(codes, scales, codes, scales, s["kv_len"], s["k_cache"], s["v_cache"], s["ws"])
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_ERR_INVALID_ARG
    assert torch.equal(s["k_cache"][1:3], k0[1:3]) and torch.all(s["k_cache"][3] == 1)


def test_no_tokens_is_a_noop(fm, cuda_device):
    s = batch(cuda_device, [(0, 0)], 2, 1, 64, 8, seed=6)
    n0 = fm.fmlp_kernel_launch_count()
    fm.fmlp_rope_append(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], fm.FmlpRope(1e4, 64), s["q_out"], s["k_cache"],
                        s["v_cache"], s["ws"])
    assert fm.fmlp_kernel_launch_count() == n0


def test_many_sequences(fm, cuda_device):
    """More sequences than one search step or one block of lengths covers, empty ones among them."""
    lens = [((i * 7) % 4, 4 + i % 3) for i in range(1500)]
    s = batch(cuda_device, lens, 2, 1, 64, 8, seed=7, behind=5)
    rot = dict(theta=1e4, rotary_dim=64)
    fm.fmlp_rope_append(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], fm.FmlpRope(**rot), s["q_out"], s["k_cache"],
                        s["v_cache"], s["ws"])
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    got = dec(s["q_out"])
    for t, r in enumerate(reference(s, rot, False, "q")):
        assert np.all(got[t] == 7) if r is None else np.all(np.abs(got[t] - r[0]) <= 2.0 ** -8 * np.abs(r[0]) + r[1])
    codes = torch.randint(-127, 128, (1500, 1, 8, 64), dtype=torch.int8, device=cuda_device)
    scales = torch.rand(1500, 1, 8, device=cuda_device)
    out = torch.zeros(1500, 1, 8, 64, dtype=torch.bfloat16, device=cuda_device)
    fm.fmlp_kv_read_q8(codes, scales, codes, scales, s["kv_len"], out, s["v_cache"], s["ws"])
    held = (torch.arange(8, device=cuda_device) < s["kv_len"][:, None])[:, None, :, None]
    assert torch.equal(out, torch.where(held, (codes.float() * scales[..., None]).to(torch.bfloat16), 0))


def test_captured_and_replayed_with_other_lengths(fm, cuda_device):
    s = batch(cuda_device, [(4, 4), (4, 4)], 2, 1, 64, 16, seed=8)
    rot = dict(theta=1e4, rotary_dim=64)
    call = lambda: fm.fmlp_rope_append(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], fm.FmlpRope(**rot),  # noqa: E731
                                       s["q_out"], s["k_cache"], s["v_cache"], s["ws"])
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    s["cu"].copy_(torch.tensor([0, 1, 8]))
    s["kv_len"].copy_(torch.tensor([3, 15]))
    s["cu_list"], s["len_list"] = [0, 1, 8], [3, 15]
    g.replay()
    torch.cuda.synchronize()
    got = dec(s["q_out"])
    for t, r in enumerate(reference(s, rot, False, "q")):
        assert np.all(np.abs(got[t] - r[0]) <= 2.0 ** -8 * np.abs(r[0]) + r[1])


def test_q8_rows_of_any_size(fm, cuda_device):
    """Rows from the smallest numbers to the largest: each within half a step (and 2^-15 of it) of its
    scale, rows under the smallest scale held as zeros, none NaN."""
    D, sizes = 64, [0.0, 1e-40, 1e-37, 2e-36, 1e-30, 1.0, 1e30, 3e38]
    s = batch(cuda_device, [(len(sizes), len(sizes))], 1, 1, D, len(sizes), seed=9)
    v = torch.linspace(-1, 1, D, dtype=torch.float64)[None] * torch.tensor(sizes, dtype=torch.float64)[:, None]
    s["v"] = v.to(torch.bfloat16)[:, None].to(cuda_device)
    codes = {c: torch.ones(1, 1, len(sizes), D, dtype=torch.int8, device=cuda_device) for c in "kv"}
    scales = {c: torch.ones(1, 1, len(sizes), device=cuda_device) for c in "kv"}
    fm.fmlp_rope_append_q8(s["q"].contiguous(), s["k"].contiguous(), s["v"], s["cu"], s["kv_len"], fm.FmlpRope(1e4, D),
                           s["q_out"], codes["k"], scales["k"], codes["v"], scales["v"], s["ws"])
    x, q, sc = dec(s["v"])[:, 0], codes["v"][0, 0].cpu().double().numpy(), scales["v"][0, 0].cpu().double().numpy()
    top = np.max(np.abs(x), axis=1)
    small = (top / 127).astype(np.float32) < 2.0 ** -125
    assert np.all(sc[small] == 0) and np.all(q[small] == 0)
    assert small.sum() == 4                      # 0, 1e-40, 1e-37, 2e-36: under 127 * 2^-125 = 2.98e-36
    err = np.abs(q * sc[:, None] - x)[~small]
    assert np.all(err <= (0.5 + 2.0 ** -15) * sc[~small][:, None]) and np.all(np.isfinite(sc))
    assert np.all(np.max(np.abs(q[~small]), axis=1) == 127)
