"""fmlp_rope_append_q8's codes, exactly: rows that are copied (v, and k without rotation) have no
rounding before them, so scale and codes are the oracle's, rint(max |x| / 127) and rint(x / s) of
the true quotients, to the last bit.  (x and s have 24 bits, so a quotient that is no half is
2^-25 away from one and binary64 tells them apart.)"""

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


def append(fm, k, v):
    """Codes and scales [n, H_kv, D] of k and v, the k rows not rotated."""
    dev, (n, H_kv, D) = k.device, k.shape
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    q = torch.zeros(n, H_kv, D, dtype=torch.bfloat16, device=dev)
    c = [torch.full((1, H_kv, n, D), 7, dtype=torch.int8, device=dev) for _ in "kv"]
    sc = [torch.full((1, H_kv, n), 7.0, device=dev) for _ in "kv"]
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    fm.fmlp_rope_append_q8(q, k, v, i32([0, n]), i32([n]), fm.FmlpRope(1e4, 0), torch.empty_like(q), c[0], sc[0], c[1],
                           sc[1], ws)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    return [(a[0].transpose(0, 1).cpu().numpy(), b[0].T.cpu().numpy()) for a, b in zip(c, sc)]


@pytest.mark.parametrize("D", [64, 96, 128])
def test_codes_of_copied_rows(fm, cuda_device, D):
    n, H_kv = 1500, 5
    x = [wl.normal_bf16(D, 90 + i, (n, H_kv, D)) for i in range(2)]
    for t, (codes, scales) in zip(x, append(fm, *(t.to(cuda_device) for t in x))):
        ref_q, ref_s = packed.quantize_kv(decode_bf16(wl.bf16_bits(t)))
        assert np.array_equal(scales, ref_s)
        assert np.array_equal(codes, ref_q)


def test_codes_next_to_a_half(fm, cuda_device):
    """Rows whose scale is a bf16 value (a maximum of 127 of them), so that halves are met exactly:
    ties go to the even code; the values beside them do not."""
    D, rows = 128, []
    for e in (-60, -3, 0, 5, 80):
        for m in (1.0, 1.25, 1.9921875):                          # 127 * m is a bf16 value for m = 1 only
            s = m * 2.0 ** e
            x = torch.zeros(D, dtype=torch.float64)
            x[0] = 127 * s
            h = torch.arange(D - 1, dtype=torch.float64) - 63.5   # halves from -63.5 on
            x[1:] = h * s
            rows.append(x.to(torch.bfloat16))
            rows.append((x * (1 + 2.0 ** -8)).to(torch.bfloat16))
            rows.append((-x * (1 - 2.0 ** -8)).to(torch.bfloat16))
    t = torch.stack(rows)[:, None]
    codes, scales = append(fm, t.to(cuda_device), t.to(cuda_device))[1]
    ref_q, ref_s = packed.quantize_kv(decode_bf16(wl.bf16_bits(t)))
    assert np.array_equal(scales, ref_s) and np.array_equal(codes, ref_q)
    x = decode_bf16(wl.bf16_bits(t))
    tie = np.abs(x / ref_s[..., None].astype(np.float64)) % 1 == 0.5
    assert tie.sum() > 100 and np.all(codes[tie] % 2 == 0)
