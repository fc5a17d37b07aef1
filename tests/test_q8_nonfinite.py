"""A NaN or an infinity that reaches the int8 side stays visible: codes cannot hold it, so the
scales and the outputs say NaN, and what does not depend on it keeps its bits."""

import math

import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def fm(cuda_device):
    import token_phase_swiglu_b200 as fm
    return fm


def setup(fm, dev, lens, H, H_kv, D, n_max, seed):
    B = len(lens)
    g = torch.Generator(device="cpu").manual_seed(seed)
    s = dict(q=wl.normal_bf16(seed, 80, (B, H, D)).to(dev), kv_len=torch.tensor(lens, dtype=torch.int32, device=dev),
             out=torch.full((B, H, D), 7.0, device=dev), scale=1 / math.sqrt(D),
             ws=torch.zeros(fm.fmlp_attn_q8_workspace_bytes(B, H, H_kv, D), dtype=torch.uint8, device=dev))
    for c in "kv":
        s[c + "_q"] = torch.randint(-127, 128, (B, H_kv, n_max, D), dtype=torch.int8, generator=g).to(dev)
        s[c + "_s"] = ((torch.rand(B, H_kv, n_max, generator=g) + 0.5) / 64).to(dev)
    return s


def decode(fm, s):
    fm.fmlp_attn_decode_q8(s["q"], s["k_q"], s["k_s"], s["v_q"], s["v_s"], s["kv_len"], s["scale"], s["out"], s["ws"])
    assert fm.fmlp_device_status(s["ws"]) == fm.FMLP_OK
    return s["out"].clone()


DECODE = [
    # lens, H, H_kv, D, n_max
    ([1, 60], 2, 2, 64, 60),
    ([300, 129, 0], 4, 2, 96, 300),
    ([200, 77], 8, 2, 128, 256),
    ([9000], 8, 1, 128, 9000),              # one region over many CTAs
    ([500, 128], 32, 2, 64, 512),
]


@pytest.mark.parametrize("lens,H,H_kv,D,n_max", DECODE)
def test_query(fm, cuda_device, lens, H, H_kv, D, n_max):
    s = setup(fm, cuda_device, lens, H, H_kv, D, n_max, seed=H + D)
    want = decode(fm, s)
    assert torch.all(torch.isfinite(want))
    clean = s["q"].clone()
    for i, bad in enumerate((NAN, INF, -INF, NAN)):
        b, h, d = i % len(lens), (3 * i + 1) % H, (37 * i + 5) % D
        s["q"].copy_(clean)
        s["q"][b, h, d] = bad
        if i == 3:
            s["q"][b, h] = NAN
        got = decode(fm, s)
        if lens[b]:
            assert torch.all(torch.isnan(got[b, h]))
            got[b, h] = want[b, h]
        assert torch.equal(got, want)


@pytest.mark.parametrize("lens,H,H_kv,D,n_max", DECODE)
@pytest.mark.parametrize("which", ["k_s", "v_s"])
def test_row_scale(fm, cuda_device, lens, H, H_kv, D, n_max, which):
    """A NaN scale of a held row: NaN for the heads that see it; of a row behind, nothing."""
    s = setup(fm, cuda_device, lens, H, H_kv, D, n_max, seed=H + D + 1)
    want = decode(fm, s)
    clean, group = s[which].clone(), H // H_kv
    for b, n in enumerate(lens):
        for row in sorted({0, n // 2, n - 1, n, n_max - 1} & set(range(n_max))):
            g = (b + row) % H_kv
            s[which].copy_(clean)
            s[which][b, g, row] = NAN
            got = decode(fm, s)
            if row < n:
                assert torch.all(torch.isnan(got[b, g * group:(g + 1) * group]))
                got[b, g * group:(g + 1) * group] = want[b, g * group:(g + 1) * group]
            assert torch.equal(got, want)


@pytest.mark.parametrize("D,R,norms", [(64, 64, False), (96, 48, True), (128, 128, False), (128, 0, True)])
def test_append(fm, cuda_device, D, R, norms):
    """A value of k or v that is not finite: its row's scale is NaN, the other rows keep their bits;
    read back and attended to, the row is NaN."""
    H, H_kv, n, held = 4, 2, 6, 9
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    x = {c: wl.normal_bf16(D, 81 + i, (n, h, D)).to(cuda_device) for i, (c, h) in enumerate((("q", H), ("k", H_kv), ("v", H_kv)))}
    gamma = wl.normal_bf16(D, 84, (D,), mean=1.0, std=0.2).to(cuda_device) if norms else None
    ws = torch.zeros(fm.fmlp_attn_q8_workspace_bytes(1, H, H_kv, D), dtype=torch.uint8, device=cuda_device)

    def append(**kw):
        a, q_out = x | kw, torch.zeros(n, H, D, dtype=torch.bfloat16, device=cuda_device)
        c = {"k_q": torch.ones(1, H_kv, held, D, dtype=torch.int8, device=cuda_device),
             "v_q": torch.ones(1, H_kv, held, D, dtype=torch.int8, device=cuda_device),
             "k_s": torch.ones(1, H_kv, held, device=cuda_device), "v_s": torch.ones(1, H_kv, held, device=cuda_device)}
        fm.fmlp_rope_append_q8(a["q"], a["k"], a["v"], i32([0, n]), i32([held]), fm.FmlpRope(1e4, R), q_out, c["k_q"],
                               c["k_s"], c["v_q"], c["v_s"], ws, q_gamma=gamma, k_gamma=gamma)
        assert fm.fmlp_device_status(ws) == fm.FMLP_OK
        return q_out, c

    q_out, want = append()
    assert all(torch.all(torch.isfinite(t)) for t in (q_out, want["k_s"], want["v_s"]))
    big = 3e38                                                    # a pair of them may turn past the largest number
    for which in "kv":
        for i, bad in enumerate((NAN, INF, -INF, big)):
            t, g, d = (2 * i + 1) % n, i % H_kv, (29 * i + 3) % D
            y = x[which].clone()
            y[t, g, d] = bad
            if bad == big:
                y[t, g] = big
            q2, got = append(**{which: y})
            row = held - n + t
            seen = which == "k" or bad != big                     # a row of v is copied, and 3e38 / 127 is a scale
            if which == "k" and bad == big:
                seen = bool(torch.isnan(got["k_s"][0, g, row]))   # by its angles
                assert seen or torch.isfinite(got["k_s"][0, g, row])
            assert torch.equal(q2, q_out)
            assert bool(torch.isnan(got[which + "_s"][0, g, row])) == seen
            bf = {c: torch.zeros(1, H_kv, held, D, dtype=torch.bfloat16, device=cuda_device) for c in "kv"}
            fm.fmlp_kv_read_q8(got["k_q"], got["k_s"], got["v_q"], got["v_s"], i32([held]), bf["k"], bf["v"], ws)
            assert bool(torch.all(torch.isnan(bf[which][0, g, row]))) == seen
            out = torch.zeros(1, H, D, device=cuda_device)
            fm.fmlp_attn_decode_q8(q_out[-1:], got["k_q"], got["k_s"], got["v_q"], got["v_s"], i32([held]),
                                   1 / math.sqrt(D), out, ws)
            if seen:
                assert torch.all(torch.isnan(out[0].view(H_kv, -1)[g])) and torch.all(torch.isfinite(out[0].view(H_kv, -1)[1 - g]))
            for c in want:                                        # the other rows
                a, b = got[c].clone(), want[c].clone()
                if c[0] == which:
                    a[0, g, row], b[0, g, row] = 0, 0
                assert torch.equal(a, b)


def test_append_query(fm, cuda_device):
    """q is not quantised: NaN and infinity stay where the rotation puts them."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    q = torch.ones(2, 2, 64, dtype=torch.bfloat16, device=cuda_device)
    q[0, 1, 3], q[1, 0, 40] = NAN, INF
    k = torch.ones(2, 1, 64, dtype=torch.bfloat16, device=cuda_device)
    c = [torch.zeros(1, 1, 2, 64, dtype=torch.int8, device=cuda_device) for _ in range(2)]
    sc = [torch.zeros(1, 1, 2, device=cuda_device) for _ in range(2)]
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_device)
    out = torch.zeros_like(q)
    fm.fmlp_rope_append_q8(q, k, k, i32([0, 2]), i32([2]), fm.FmlpRope(1e4, 64), out, c[0], sc[0], c[1], sc[1], ws)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 1, [3, 35]] = True
    want[1, 0, [8, 40]] = True
    assert torch.equal(bad, want) and all(torch.all(torch.isfinite(t)) for t in sc)
