"""fmlp_attn_decode_q8 is of f32 precision: element bounds from its roundings, an order of
magnitude under what one digit less of its split operands would give.

With s_j the base-2 score of row j, v_j = codes * scale, w_j the softmax weight, u = 2^-24 and
Q = max |q| max_j sum_d |k_jd| scale log2 e:
  * a score: queries to 2^-30 of the largest, 2^-30 Q; the digits' sums joined, the scale's and
    the two products' roundings, at most 8 u |s_j|;
  * a weight's exponent s_j + log2 vs_j less the unit's largest: log2 to 2^-22 near 1 and 2 u of
    its value elsewhere, the sum and the difference rounded: 4 u (|s_j| + |log2 vs_j|) + 2^-22;
  * exp2 to 2^-22, once for the weight, once for each joining of units, threads and pieces;
so w_j is off by w_j e_j with e_j = ln 2 (2^-30 Q + u (12 |s_j| + 4 |log2 vs_j|) + 2^-22) + 2^-21,
in the numerator and in the sum l.  Sums in f32 over units and pieces: 2^-19 of their terms, for
the few tens of units a CTA has here.  The digits of a weight hold it to 2^-25 of the unit's
largest |weight * vs|, 128 rows a unit, codes up to 127: 2^-18 of max_j w_j 127 vs_j at most.  So
  |o - o_ref| <= sum_j w_j e_j (|v_j| + |o|) + 2^-19 (sum_j w_j |v_j| + |o|) + 2^-18 max_j w_j 127 vs_j.

The first tests hold the bound to an emulation of the kernel's arithmetic on the CPU: it passes with
the digits that the kernel takes and fails with one digit of the weights less, or with three digits
of base 128 for a query with an outlier."""

import math

import numpy as np
import pytest
import torch

from oracle import decode_bf16
import workloads as wl

U = 2.0 ** -24
LOG2E = math.log2(math.e)


def problem(lens, H, H_kv, D, n_max, seed, outlier=0.0, std=2.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    B = len(lens)
    q = wl.normal_bf16(seed, 95, (B, H, D), std=std)
    k_q, v_q = (torch.randint(-127, 128, (B, H_kv, n_max, D), dtype=torch.int8, generator=g) for _ in range(2))
    k_s, v_s = ((torch.rand(B, H_kv, n_max, generator=g) + 0.5) / 64 for _ in range(2))
    if outlier:                                   # one channel far above the rest, where keys are (almost) nothing
        q[..., 5] = outlier
        k_q[..., 5] = 0
        k_q[:, :, ::7, 5] = 1
        k_s[:, :, ::7] /= outlier
    return dict(q=q, k_q=k_q, k_s=k_s, v_q=v_q, v_s=v_s, lens=lens, scale=1 / math.sqrt(D))


def exact_and_bound(p, b, h):
    H_kv, L = p["k_q"].shape[1], p["lens"][b]
    g = h // (p["q"].shape[1] // H_kv)
    q = decode_bf16(wl.bf16_bits(p["q"]))[b, h]
    K = p["k_q"][b, g, :L].numpy().astype(np.float64) * p["k_s"][b, g, :L, None].numpy().astype(np.float64)
    vs = p["v_s"][b, g, :L].numpy().astype(np.float64)
    V = p["v_q"][b, g, :L].numpy().astype(np.float64) * vs[:, None]
    s = K @ q * (p["scale"] * LOG2E)
    w = np.exp2(s - s.max())
    w /= w.sum()
    o = w @ V
    Q = np.max(np.abs(q)) * np.max(np.sum(np.abs(K), axis=1)) * p["scale"] * LOG2E
    e = math.log(2) * (2.0 ** -30 * Q + U * (12 * np.abs(s) + 4 * np.abs(np.log2(vs))) + 2.0 ** -22) + 2.0 ** -21
    bound = (w * e) @ (np.abs(V) + np.abs(o)) + 2.0 ** -19 * (w @ np.abs(V) + np.abs(o)) + 2.0 ** -18 * np.max(w * 127 * vs)
    return o, bound


def emulate(p, b, h, digits_q=4, base_q=256, digits_w=3):
    """The kernel's arithmetic for one region held by one CTA: f32 throughout."""
    f = np.float32
    H_kv, L = p["k_q"].shape[1], p["lens"][b]
    g = h // (p["q"].shape[1] // H_kv)
    q = decode_bf16(wl.bf16_bits(p["q"]))[b, h]
    kq, vq = (p[c][b, g, :L].numpy().astype(np.int64) for c in ("k_q", "v_q"))
    ks, vs = (p[c][b, g, :L].numpy() for c in ("k_s", "v_s"))
    bits = 29 if base_q == 256 else 5 + 7 * (digits_q - 1)
    top = 2.0 ** (bits - math.floor(math.log2(np.max(np.abs(q)))))
    x = np.rint(q * top).astype(np.int64)
    low = base_q ** (digits_q - 1) if base_q == 128 else 2 ** 24
    joined = (kq @ x / low).astype(f)             # exact sums, one rounding
    s = joined * f(low / top * p["scale"] * LOG2E) * ks
    ex = s + np.log2(vs).astype(f)
    acc, ref, m, l = np.zeros(vq.shape[1], f), f(-np.inf), f(-np.inf), f(0)
    for j in range(0, L, 128):
        t = ex[j:j + 128].max()
        y = f(127) * np.exp2(ex[j:j + 128] - t, dtype=f)
        total = np.zeros(vq.shape[1])
        for i in range(digits_w):
            d = np.rint(y)
            assert np.all(np.abs(d) <= 127)
            total = total + (d.astype(np.int64) @ vq[j:j + 128]) / 254.0 ** i
            y = (y - d) * f(254)
        n = max(ref, t)
        acc = acc * np.exp2(ref - n, dtype=f) + total.astype(f) * np.exp2(t - n, dtype=f)
        ref = n
        mn = max(m, s[j:j + 128].max())
        l = l * np.exp2(m - mn, dtype=f) + np.exp2(s[j:j + 128] - mn, dtype=f).sum(dtype=f)
        m = mn
    return (acc * np.exp2(ref - m, dtype=f) / (f(127) * l)).astype(np.float64)


def ratio(p, got):
    worst = 0.0
    for b, L in enumerate(p["lens"]):
        for h in range(p["q"].shape[1] if L else 0):
            o, bound = exact_and_bound(p, b, h)
            worst = max(worst, float(np.max(np.abs(got(b, h) - o) / bound)))
    return worst


CASES = [
    # lens, H, H_kv, D, n_max
    ([5], 4, 2, 64, 8),
    ([128], 1, 1, 128, 128),
    ([129, 127, 1, 0, 256], 8, 2, 128, 256),
    ([1000], 32, 8, 128, 1001),
    ([300, 77], 12, 4, 96, 301),
    ([333], 7, 1, 64, 334),
    ([400, 90], 16, 1, 128, 512),
    ([260] * 3, 18, 2, 96, 260),
    ([700], 16, 16, 64, 700),
    ([900, 31], 4, 4, 96, 900),
]
OUTLIERS = [24.0, 1000.0, 65536.0, -2.0 ** 20]


@pytest.mark.parametrize("lens,H,H_kv,D,n_max", CASES)
def test_bound_holds_for_the_emulation(lens, H, H_kv, D, n_max):
    p = problem(lens, H, H_kv, D, n_max, seed=H + D)
    assert ratio(p, lambda b, h: emulate(p, b, h)) <= 1
    if max(lens) > 5:
        assert ratio(p, lambda b, h: emulate(p, b, h, digits_w=2)) > 1


@pytest.mark.parametrize("outlier", OUTLIERS)
def test_bound_finds_a_coarse_query(outlier):
    p = problem([600], 8, 2, 128, 600, seed=3, outlier=outlier)
    assert ratio(p, lambda b, h: emulate(p, b, h)) <= 1
    if abs(outlier) > 100:
        assert ratio(p, lambda b, h: emulate(p, b, h, digits_q=3, base_q=128)) > 1


@pytest.fixture(scope="module")
def fm(cuda_device):
    import token_phase_swiglu_b200 as fm
    return fm


def run(fm, dev, p):
    B, H, D = p["q"].shape
    n = {c: p[c].to(dev) for c in ("q", "k_q", "k_s", "v_q", "v_s")}
    ws = torch.zeros(fm.fmlp_attn_q8_workspace_bytes(B, H, p["k_q"].shape[1], D), dtype=torch.uint8, device=dev)
    out = torch.empty(B, H, D, device=dev)
    fm.fmlp_attn_decode_q8(n["q"], n["k_q"], n["k_s"], n["v_q"], n["v_s"],
                           torch.tensor(p["lens"], dtype=torch.int32, device=dev), p["scale"], out, ws)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    return out.cpu().double().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,H_kv,D,n_max", CASES)
def test_every_digit_counts(fm, cuda_device, lens, H, H_kv, D, n_max):
    p = problem(lens, H, H_kv, D, n_max, seed=H + D)
    got = run(fm, cuda_device, p)
    worst = ratio(p, lambda b, h: got[b, h])
    print(f"of the bound: {worst:.2f}")
    assert worst <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("H,H_kv,D", [(8, 2, 128), (2, 2, 64), (16, 1, 96), (8, 1, 64), (4, 2, 96)])
@pytest.mark.parametrize("outlier", OUTLIERS)
def test_query_with_an_outlier(fm, cuda_device, outlier, H, H_kv, D):
    p = problem([600], H, H_kv, D, 600, seed=3, outlier=outlier)
    got = run(fm, cuda_device, p)
    assert ratio(p, lambda b, h: got[b, h]) <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** -125, 2.0 ** -100, 2.0 ** -97, 2.0 ** -20, 2.0 ** 60])
def test_queries_of_any_size(fm, cuda_device, size):
    """The scale that undoes the queries' size leaves the scores as they were (under 2^-98 a query is
    held to 2^-128, which is 2^-3 of the smallest here: only its sign and size are asked for)."""
    p = problem([300], 8, 2, 128, 300, seed=4)
    q = decode_bf16(wl.bf16_bits(p["q"])) / 16
    p["q"] = torch.from_numpy(q * size).to(torch.bfloat16)
    p["k_s"] = p["k_s"] * (2.0 ** 60 if size < 1 else 2.0 ** -30)
    p["scale"] = min(1 / size / math.sqrt(128) * (2.0 ** -60 if size < 1 else 2.0 ** 30), 2.0 ** 120)
    got = run(fm, cuda_device, p)
    if size >= 2.0 ** -97:
        assert ratio(p, lambda b, h: got[b, h]) <= 1
    else:
        assert np.all(np.isfinite(got))
