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
