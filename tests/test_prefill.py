"""fmlp_attn_prefill against the binary64 oracle.

Tolerance.  Inputs are bf16, so the products q k are exact in f32 and a score is
off by its f32 sums (relative 2^-24 a term) only.  Each softmax weight is rounded
to bf16 (half a step: 2^-8 of it at most) for its product with V while the sum l
takes it unrounded, so |o - o_ref| <= 2^-8 sum_j w_j |v_j| / l; the result is
rounded to bf16 (2^-8 |o|); scores up to 2^6 in base 2 with the hardware exp2 and
f32 sums add less than 2^-12 of the same sum.  Every element is asked to be
within 2^-8 (|o| + A) + 2^-11 A, A = sum_j w_j |v_j| / l."""

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


def dec(t):
    return decode_bf16(wl.bf16_bits(t.detach().cpu()))


def setup(fm, dev, lens, H, H_kv, D, n_max, seed, front=0, behind=0, std=2.0):
    cu = [front]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    T, B = cu[-1] + behind, len(lens)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(q=wl.normal_bf16(seed, 50, (T, H, D), std=std).to(dev), cu=i32(cu), kv_len=i32([x for _, x in lens]),
             k=wl.normal_bf16(seed, 51, (B, H_kv, n_max, D)).to(dev),
             v=wl.normal_bf16(seed, 52, (B, H_kv, n_max, D)).to(dev), cu_list=cu, len_list=[x for _, x in lens],
             out=torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=dev), scale=1 / math.sqrt(D),
             ws=torch.zeros(fm.fmlp_prefill_workspace_bytes(T, B, H, H_kv, D), dtype=torch.uint8, device=dev))
    for b, (_, held) in enumerate(lens):  # the rows behind a sequence hold anything
        s["k"][b, :, max(held, 0):] = float("nan")
        s["v"][b, :, max(held, 0):] = float("inf")
    return s


def call(fm, s):
    fm.fmlp_attn_prefill(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], s["scale"], s["out"], s["ws"])


def reference(s, rows=None):
    """o and A of every token (NaN where nothing is written), by the oracle."""
    q, k, v = dec(s["q"]), dec(s["k"]), dec(s["v"])
    o = packed.causal_attention(q, k, v, s["cu_list"], s["len_list"], s["scale"])
    a = packed.causal_attention(q, k, np.abs(v), s["cu_list"], s["len_list"], s["scale"])
    return o, a


def check(s, got=None):
    o, a = reference(s)
    got = dec(s["out"]) if got is None else got
    written = ~np.isnan(o[:, 0, 0])
    assert np.all(got[~written] == 7.0)
    d = np.abs(got[written] - o[written])
    bound = 2.0 ** -8 * (np.abs(o[written]) + a[written]) + 2.0 ** -11 * a[written]
    assert np.all(d <= bound), float(np.max(d - bound))
    return float(np.linalg.norm(d) / max(np.linalg.norm(o[written]), 1e-30))


CASES = [
    # lens (new, held), H, H_kv, D, n_max
    ([(1, 1)], 1, 1, 64, 1),
    ([(1, 5)], 4, 2, 64, 8),
    ([(128, 128)], 1, 1, 128, 128),
    ([(129, 129)], 2, 2, 128, 130),
    ([(300, 300)], 2, 1, 64, 301),
    ([(65, 65)], 8, 2, 128, 77),
    ([(40, 40)], 12, 4, 96, 64),                               # 3 heads per KV head: 126 rows a tile
    ([(7, 260), (1, 128), (0, 9), (33, 129), (2, 2)], 8, 1, 128, 300),
    ([(1, 1000), (1, 1), (1, 513)], 40, 8, 128, 1000),           # 5 heads per KV head, one token each
    ([(4, 777)] * 6, 32, 8, 128, 800),                           # draft tokens
    ([(200, 200), (90, 350)], 3, 3, 96, 400),
    ([(1, 3000)], 16, 16, 64, 3001),                             # one token, split over many CTAs
    ([(3, 4000)], 16, 1, 64, 4096),                              # 16 heads per KV head
    ([(2, 50)], 128, 1, 64, 64),                                 # 128 heads per KV head: one token a tile
    ([(9, 40)], 100, 1, 96, 64),
    ([(4, 2), (3, 0), (200, 60), (2, 2)], 4, 2, 64, 64),         # padding: fewer rows than new tokens
    ([(600, 600), (1, 900)], 2, 2, 128, 900),
]


@pytest.mark.parametrize("lens,H,H_kv,D,n_max", CASES)
def test_prefill_matches_oracle(fm, cuda_device, lens, H, H_kv, D, n_max):
    s = setup(fm, cuda_device, lens, H, H_kv, D, n_max, seed=len(lens) + H * 3 + D, front=2, behind=3)
    n0 = fm.fmlp_kernel_launch_count()
    call(fm, s)
    assert fm.fmlp_kernel_launch_count() == n0 + 1
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    print(f"normwise {check(s):.2e}")
    first = s["out"].clone()
    s["out"].fill_(7.0)
    call(fm, s)                                                  # the workspace is ready again
    assert torch.equal(s["out"], first)                          # and the result the same


def test_growing_scores_rescale(fm, cuda_device):
    """Keys that grow along the sequence push the running maximum up by more than the lazy
    reference allows, tile after tile; shrinking ones never do."""
    for order in (1, -1):
        s = setup(fm, cuda_device, [(5, 700), (256, 700)], 4, 2, 64, 700, seed=9)
        size = torch.linspace(0.05, 4, 700, device=cuda_device)[:: order or 1] if order > 0 else \
            torch.linspace(4, 0.05, 700, device=cuda_device)
        s["k"] = (s["k"].float() * size[:, None]).to(torch.bfloat16)
        call(fm, s)
        assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
        check(s)


def test_equal_scores_and_far_below(fm, cuda_device):
    """Zero queries average the rows; scores of -10^4 and less underflow to nothing but the maximum."""
    s = setup(fm, cuda_device, [(140, 400)], 2, 2, 64, 400, seed=10)
    s["q"][:70] = 0
    s["q"][70:] *= 64
    call(fm, s)
    check(s)


def test_strided_queries(fm, cuda_device):
    s = setup(fm, cuda_device, [(70, 70), (3, 200)], 4, 2, 96, 200, seed=11)
    call(fm, s)
    want = s["out"].clone()
    wide = torch.full((73, 8 * 96), 5.0, dtype=torch.bfloat16, device=cuda_device)
    wide[:, 96:5 * 96] = s["q"].flatten(1)
    s["q"] = wide[:, 96:5 * 96].unflatten(1, (4, 96))
    call(fm, s)
    assert torch.equal(s["out"], want)


def test_many_sequences(fm, cuda_device):
    """More sequences than a block has threads, empty ones among them."""
    lens = [((i * 5) % 4, (i * 5) % 4 + i % 50) for i in range(900)]
    s = setup(fm, cuda_device, lens, 2, 1, 64, 64, seed=12, behind=1)
    call(fm, s)
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    check(s)


def test_no_work_at_all(fm, cuda_device):
    s = setup(fm, cuda_device, [(0, 5), (0, 0)], 2, 1, 64, 64, seed=13, behind=4)
    call(fm, s)
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    assert torch.all(s["out"] == 7)


def test_bad_lengths(fm, cuda_device):
    """A length past n_max, a negative one, a range past T: reported, left alone, the others done."""
    s = setup(fm, cuda_device, [(3, 3), (5, 20), (4, 30)], 4, 2, 64, 64, seed=14)
    s["kv_len"].copy_(torch.tensor([3, 65, 30]))
    call(fm, s)
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_ERR_INVALID_ARG
    assert torch.all(s["out"][3:8] == 7)
    got = dec(s["out"])
    s["kv_len"].copy_(torch.tensor([3, 20, 30]))
    o, a = reference(s)
    for t in list(range(3)) + list(range(8, 12)):
        assert np.all(np.abs(got[t] - o[t]) <= 2.0 ** -8 * (np.abs(o[t]) + a[t]) + 2.0 ** -11 * a[t])
    for kv, cu in (([3, -1, 30], [0, 3, 8, 12]), ([3, 20, 30], [0, 3, 8, 13]), ([3, 20, 30], [0, 3, 2, 12])):
        s["kv_len"].copy_(torch.tensor(kv))
        s["cu"].copy_(torch.tensor(cu))
        call(fm, s)
        assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_ERR_INVALID_ARG


def test_captured_graphs_share_a_workspace(fm, cuda_device):
    """Two calls of other shapes captured with one workspace, replayed in turn with other lengths."""
    a = setup(fm, cuda_device, [(3, 700), (2, 300)], 8, 2, 64, 700, seed=15)
    b = setup(fm, cuda_device, [(200, 200)], 4, 4, 128, 260, seed=16)
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
    a["cu"].copy_(torch.tensor([0, 1, 5]))
    a["kv_len"].copy_(torch.tensor([650, 299]))
    a["cu_list"], a["len_list"] = [0, 1, 5], [650, 299]
    for s in (a, b):
        s["out"].fill_(7.0)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    check(a)
    check(b)


def test_on_another_stream(fm, cuda_device):
    s = setup(fm, cuda_device, [(50, 90)], 4, 2, 128, 90, seed=17)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        call(fm, s)
    st.synchronize()
    check(s)


def test_bounded_waits(fm, cuda_device):
    """Each CTA's last tile withheld (host-side fault injection): the waits expire, the call reports
    FMLP_ERR_TIMEOUT and, the workspace zeroed, the next one is right."""
    s = setup(fm, cuda_device, [(300, 900), (5, 800)], 8, 2, 128, 900, seed=18)
    try:
        fm.fmlp_set_wait_timeout_ns(2_000_000)
        fm.fmlp_set_fault_injection(1)
        call(fm, s)
        assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_ERR_TIMEOUT
    finally:
        fm.fmlp_set_fault_injection(0)
        fm.fmlp_set_wait_timeout_ns(0)
    s["ws"].zero_()
    s["out"].fill_(7.0)
    call(fm, s)
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    check(s)


def test_far_into_a_large_cache(fm, cuda_device):
    """Offsets past 2^31 elements of the cache (the last region of a 6 GB cache)."""
    B, H_kv, n_max, D = 12, 8, 262144, 128
    k = torch.zeros(B, H_kv, n_max, D, dtype=torch.bfloat16, device=cuda_device)
    v = torch.zeros_like(k)
    k[-1, -1, :260000] = torch.randn(260000, D, device=cuda_device).to(torch.bfloat16)
    v[-1, -1, :260000] = torch.randn(260000, D, device=cuda_device).to(torch.bfloat16)
    q = (2 * torch.randn(2, 16, D, device=cuda_device)).to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    cu, kv_len = i32([0] * B + [2]), i32([0] * (B - 1) + [260000])
    out = torch.empty_like(q)
    ws = torch.zeros(fm.fmlp_prefill_workspace_bytes(2, B, 16, H_kv, D), dtype=torch.uint8, device=cuda_device)
    fm.fmlp_attn_prefill(q, k, v, cu, kv_len, 1 / math.sqrt(D), out, ws)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    for t in range(2):
        n = 260000 - 1 + t
        z = torch.softmax(k[-1, -1, :n].double() @ q[t, 14:].double().T / math.sqrt(D), 0)
        o, a = z.T @ v[-1, -1, :n].double(), z.T @ v[-1, -1, :n].double().abs()
        assert torch.all((out[t, 14:].double() - o).abs() <= 2.0 ** -8 * (o.abs() + a) + 2.0 ** -11 * a)
