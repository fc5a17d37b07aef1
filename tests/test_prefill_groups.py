"""fmlp_attn_prefill's schedule for every shape of a query tile: from 1 to 128 heads a KV head, prompts
of many tiles, continued and padded ones, split over the CTAs by a closed form of the units before
each pair of tiles.  A share that starts in the wrong place leaves rows out or takes them twice, so
the outputs are compared element by element with binary64 (2^-8 (|o| + A) + 2^-11 A as in the other
tests of this call)."""

import math

import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 9, 11, 16, 27, 33, 64, 100, 128])
def test_heads_per_kv_head(cuda_device, G):
    import token_phase_swiglu_b200 as fm
    H_kv, D, per = 2, 64, 2 * (128 // G)                     # tokens of a pair of tiles
    n = min(9 * per + per // 2 + 1, 2048 // G + 60)
    lens = [(n, n), (per, 3 * per + 77), (n + 3, n - per - 1), (1, 500), (n, n + 1000)]
    H, B, cu = G * H_kv, len(lens), [0]
    for x, _ in lens:
        cu.append(cu[-1] + x)
    T, n_max = cu[-1], max(x for _, x in lens)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    q = wl.normal_bf16(G, 120, (T, H, D), std=2.0).to(cuda_device)
    k, v = (wl.normal_bf16(G, 121 + i, (B, H_kv, n_max, D)).to(cuda_device) for i in range(2))
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=cuda_device)
    ws = torch.zeros(fm.fmlp_prefill_workspace_bytes(T, B, H, H_kv, D), dtype=torch.uint8, device=cuda_device)
    fm.fmlp_attn_prefill(q, k, v, i32(cu), i32([x for _, x in lens]), 1 / math.sqrt(D), out, ws)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    for b, (new, held) in enumerate(lens):
        K, V = (t[b, :, :max(held, 0)].double().repeat_interleave(G, 0) for t in (k, v))
        rows = torch.arange(held - new, held, device=cuda_device)        # each token's position
        x = q[cu[b]:cu[b + 1]].double().transpose(0, 1)
        z = (x @ K.mT / math.sqrt(D)).masked_fill(torch.arange(held, device=cuda_device) > rows[:, None], -math.inf)
        w = torch.nan_to_num(torch.softmax(z, -1))                       # padding tokens see no row: zeros
        o, a = w @ V, w @ V.abs()
        got = out[cu[b]:cu[b + 1]].double().transpose(0, 1)
        assert torch.all((got - o).abs() <= 2.0 ** -8 * (o.abs() + a) + 2.0 ** -11 * a), b
