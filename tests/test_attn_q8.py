"""fmlp_attn_decode_q8 against the binary64 oracle, on the same codes and scales.

Tolerance.  Codes are multiplied exactly.  A query value is held to 2^-20 of its
head's largest |q|, so with Q = max|q| max_j sum_d |k_jd| scale, a score is off by at
most 2^-20 Q plus f32 roundings of the joined sums and products (8 of 2^-24 of |s|,
|s| <= Q): under 1.5 * 2^-20 Q.  That moves a weight by as much, relatively, in the
numerator and in l; the hardware's exp2 and log2 add 2^-21 each time.  Weights are held
to 2^-24 of their unit's largest, 128 rows a unit.  With W = sum_j w_j |v_j| / l:
|o - o_ref| <= (3 * 2^-20 Q + 2^-19) W + 2^-17 max_j |w_j v_j| / l; the test asks for
2^-18 (1 + Q) W + 2^-15 max_j |w_j v_j| / l."""

import math

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


def setup(fm, dev, lens, H, H_kv, D, n_max, seed, std=2.0):
    B = len(lens)
    g = torch.Generator(device="cpu").manual_seed(seed)
    s = dict(q=wl.normal_bf16(seed, 60, (B, H, D), std=std).to(dev),
             kv_len=torch.tensor(lens, dtype=torch.int32, device=dev), lens=lens, scale=1 / math.sqrt(D),
             out=torch.full((B, H, D), 7.0, device=dev),
             ws=torch.zeros(fm.fmlp_attn_q8_workspace_bytes(B, H, H_kv, D), dtype=torch.uint8, device=dev))
    for c in "kv":
        s[c + "_q"] = torch.randint(-127, 128, (B, H_kv, n_max, D), dtype=torch.int8, generator=g).to(dev)
        s[c + "_s"] = ((torch.rand(B, H_kv, n_max, generator=g) + 0.5) / 64).to(dev)
        for b, n in enumerate(lens):   # rows behind a sequence hold anything
            s[c + "_s"][b, :, max(n, 0):] = float("nan")
    return s


def call(fm, s):
    fm.fmlp_attn_decode_q8(s["q"], s["k_q"], s["k_s"], s["v_q"], s["v_s"], s["kv_len"], s["scale"], s["out"], s["ws"])


def check(s, skip=()):
    n = {c: s[c].cpu().numpy() for c in ("k_q", "k_s", "v_q", "v_s")}
    q, got = decode_bf16(wl.bf16_bits(s["q"].cpu())), s["out"].cpu().double().numpy()
    lens = [0 if b in skip else x for b, x in enumerate(s["lens"])]
    o = packed.decode_attention_q8(q, n["k_q"], n["k_s"], n["v_q"], n["v_s"], lens, s["scale"])
    W = packed.decode_attention_q8(q, n["k_q"], n["k_s"], np.abs(n["v_q"].astype(np.int16)), n["v_s"], lens, s["scale"])
    B, H, D = q.shape
    group = H // n["k_q"].shape[1]
    worst = 0.0
    for b, L in enumerate(lens):
        if b in skip:
            assert np.all(got[b] == 7.0)
            continue
        if L == 0:
            assert np.all(got[b] == 0.0)
            continue
        for h in range(H):
            K = n["k_q"][b, h // group, :L].astype(np.float64) * n["k_s"][b, h // group, :L, None]
            V = n["v_q"][b, h // group, :L].astype(np.float64) * n["v_s"][b, h // group, :L, None]
            z = s["scale"] * (K @ q[b, h])
            w = np.exp(z - z.max())
            Q = np.max(np.abs(q[b, h])) * np.max(np.sum(np.abs(K), axis=1)) * s["scale"]
            top = np.max(w[:, None] * np.abs(V)) / np.sum(w)
            d = np.abs(got[b, h] - o[b, h])
            assert np.all(d <= 2.0 ** -18 * (1 + Q) * W[b, h] + 2.0 ** -15 * top), (b, h, d.max())
        worst = max(worst, np.linalg.norm(got[b] - o[b]) / np.linalg.norm(o[b]))
    return worst


CASES = [
    # lens, H, H_kv, D, n_max
    ([1], 1, 1, 64, 1),
    ([5], 4, 2, 64, 8),
    ([128], 1, 1, 128, 128),
    ([129, 127, 1, 0, 256], 8, 2, 128, 256),
    ([1000], 32, 8, 128, 1001),
    ([300, 77], 12, 4, 96, 301),                    # 3 heads per KV head
    ([700, 1, 513], 40, 8, 128, 701),               # 5
    ([333], 7, 1, 64, 334),                         # 7
    ([400, 90], 16, 1, 128, 512),                   # 16
    ([260] * 3, 18, 2, 96, 260),                    # 9
    ([4096], 32, 32, 96, 4096),
    ([20000], 4, 1, 128, 20001),                    # one region over every CTA
    ([0, 0], 2, 1, 64, 4),
]


@pytest.mark.parametrize("lens,H,H_kv,D,n_max", CASES)
def test_matches_oracle(fm, cuda_device, lens, H, H_kv, D, n_max):
    s = setup(fm, cuda_device, lens, H, H_kv, D, n_max, seed=H * 7 + D + len(lens))
    n0 = fm.fmlp_kernel_launch_count()
    call(fm, s)
    assert fm.fmlp_kernel_launch_count() == n0 + 1
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    print(f"normwise {check(s):.2e}")
    first = s["out"].clone()
    call(fm, s)
    assert torch.equal(s["out"], first)


def test_rows_of_very_different_size(fm, cuda_device):
    """A row whose value scale is 10^4 times the others' (and whose weight is small), rows of
    zeros, a head of zero queries: the weights of the rest keep their precision."""
    s = setup(fm, cuda_device, [600], 8, 2, 128, 600, seed=3)
    s["v_s"][0, :, 17] = 200.0
    s["k_q"][0, :, 17] = 0
    s["v_s"][0, :, 40:60] = 0
    s["k_s"][0, :, 300] = 0
    s["q"][0, 3] = 0
    call(fm, s)
    check(s)


def test_sink_row(fm, cuda_device):
    """One row far above thousands of small ones, whose mass together is the same."""
    n, D = 8192, 64
    s = setup(fm, cuda_device, [n], 2, 1, D, n, seed=4)
    s["q"].fill_(1.0)
    s["k_q"].zero_()
    s["k_s"].fill_(1 / 127)
    s["k_q"][0, 0, 5] = 127
    s["scale"] = math.log(n) / D
    call(fm, s)
    check(s)


def test_all_values_zero(fm, cuda_device):
    s = setup(fm, cuda_device, [200], 4, 2, 64, 200, seed=5)
    s["v_s"].zero_()
    call(fm, s)
    assert torch.all(s["out"] == 0)


def test_many_sequences(fm, cuda_device):
    s = setup(fm, cuda_device, [(i * 37) % 150 for i in range(800)], 4, 2, 64, 152, seed=6)
    call(fm, s)
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    check(s)


def test_bad_lengths(fm, cuda_device):
    s = setup(fm, cuda_device, [100, 30, 40, 64], 4, 2, 64, 128, seed=7)
    s["kv_len"].copy_(torch.tensor([100, 129, -1, 64]))
    call(fm, s)
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_ERR_INVALID_ARG
    check(s, skip=(1, 2))


def test_captured_graphs_share_a_workspace(fm, cuda_device):
    a = setup(fm, cuda_device, [900, 20], 8, 2, 128, 1000, seed=8)
    b = setup(fm, cuda_device, [300], 5, 1, 96, 400, seed=9)
    ws = max(a["ws"], b["ws"], key=lambda t: t.numel())
    a["ws"] = b["ws"] = ws
    graphs = []
    for s in (a, b):
        call(fm, s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(fm, s)
        graphs.append(g)
    a["lens"] = [500, 20]
    a["kv_len"].copy_(torch.tensor(a["lens"]))
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    check(a)
    check(b)


def test_bounded_waits(fm, cuda_device):
    s = setup(fm, cuda_device, [3000, 100], 8, 2, 128, 3000, seed=10)
    try:
        fm.fmlp_set_wait_timeout_ns(2_000_000)
        fm.fmlp_set_fault_injection(1)
        call(fm, s)
        assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_ERR_TIMEOUT
    finally:
        fm.fmlp_set_fault_injection(0)
        fm.fmlp_set_wait_timeout_ns(0)
    s["ws"].zero_()
    call(fm, s)
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    check(s)


def test_far_into_a_large_cache(fm, cuda_device):
    """Offsets past 2^32 bytes: the last region of a 4.8 GB cache."""
    B, H_kv, n_max, D = 9, 16, 262144, 128
    kq = torch.zeros(B, H_kv, n_max, D, dtype=torch.int8, device=cuda_device)
    vq = torch.zeros_like(kq)
    ks = torch.zeros(B, H_kv, n_max, device=cuda_device)
    vs = torch.zeros_like(ks)
    n = 260001
    for t in (kq, vq):
        t[-1, -1, :n] = torch.randint(-127, 128, (n, D), dtype=torch.int8, device=cuda_device)
    for t in (ks, vs):
        t[-1, -1, :n] = (torch.rand(n, device=cuda_device) + 0.5) / 64
    q = torch.randn(B, 32, D, device=cuda_device).to(torch.bfloat16)
    kv_len = torch.tensor([0] * (B - 1) + [n], dtype=torch.int32, device=cuda_device)
    out = torch.full((B, 32, D), 7.0, device=cuda_device)
    ws = torch.zeros(fm.fmlp_attn_q8_workspace_bytes(B, 32, H_kv, D), dtype=torch.uint8, device=cuda_device)
    fm.fmlp_attn_decode_q8(q, kq, ks, vq, vs, kv_len, 1 / math.sqrt(D), out, ws)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    assert torch.all(out[:-1] == 0)
    K, V = (c[-1, -1, :n].double() * x[-1, -1, :n, None].double() for c, x in ((kq, ks), (vq, vs)))
    w = torch.softmax(K @ q[-1, 30:].double().T / math.sqrt(D), 0)
    o, W = w.T @ V, w.T @ V.abs()
    Q = q[-1, 30:].double().abs().amax() * K.abs().sum(1).amax() / math.sqrt(D)
    assert torch.all((out[-1, 30:].double() - o).abs() <= 2.0 ** -18 * (1 + Q) * W)
