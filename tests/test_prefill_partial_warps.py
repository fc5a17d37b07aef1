"""fmlp_attn_prefill with query rows that end inside a warp, for items that one CTA holds, items cut
between CTAs and joined by the one that holds their start or by another: element by element against
the binary64 oracle (2^-8 (|o| + A) + 2^-11 A, A = sum_j w_j |v_j| / l: weights and output rounded to
bf16 once each, the rest f32), with rows of other tokens left alone and the same bits every time."""

import math

import numpy as np
import pytest
import torch

from oracle import decode_bf16, packed
import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("lens,H,H_kv", [
    ([(5, 4000)], 3, 1),                       # 15 rows, cut over many CTAs
    ([(45, 2500)], 3, 1),                      # 126 rows and 9: a warp of 30 and one of 9
    ([(7, 900), (11, 1300), (1, 2000)], 10, 2),
    ([(50, 50), (3, 7)], 5, 1),                # not cut
    ([(129, 1100)], 7, 7),                     # one row in the second tile
])
def test_rows_that_end_inside_a_warp(cuda_device, lens, H, H_kv, D):
    import token_phase_swiglu_b200 as fm
    cu = [1]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    T, B, n_max = cu[-1] + 2, len(lens), max(x for _, x in lens)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    q = wl.normal_bf16(D, 110, (T, H, D), std=2.0)
    k, v = (wl.normal_bf16(D, 111 + i, (B, H_kv, n_max, D)) for i in range(2))
    kv_len = [x for _, x in lens]
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=cuda_device)
    ws = torch.zeros(fm.fmlp_prefill_workspace_bytes(T, B, H, H_kv, D), dtype=torch.uint8, device=cuda_device)
    args = (q.to(cuda_device), k.to(cuda_device), v.to(cuda_device), i32(cu), i32(kv_len), 1 / math.sqrt(D), out, ws)
    fm.fmlp_attn_prefill(*args)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    first = out.clone()
    for _ in range(20):
        fm.fmlp_attn_prefill(*args)
    assert torch.equal(out, first)
    qd, kd, vd = (decode_bf16(wl.bf16_bits(t)) for t in (q, k, v))
    o = packed.causal_attention(qd, kd, vd, cu, kv_len, 1 / math.sqrt(D))
    a = packed.causal_attention(qd, kd, np.abs(vd), cu, kv_len, 1 / math.sqrt(D))
    got = decode_bf16(wl.bf16_bits(out.cpu()))
    done = slice(cu[0], cu[-1])
    assert np.all(got[:cu[0]] == 7) and np.all(got[cu[-1]:] == 7)
    assert np.all(np.abs(got[done] - o[done]) <= 2.0 ** -8 * (np.abs(o[done]) + a[done]) + 2.0 ** -11 * a[done])
