"""fmlp_attn_prefill where one of a pair of query tiles has no part in some units: sequences of an odd
number of tiles, and items cut where only the second tile sees the rest, one short segment after another
in a CTA.  The two tiles' softmax groups then run ahead of each other; what one does to the shared K and V
tiles (zeroing the rows behind a sequence's end, which hold NaN and infinities here) must not reach the
other's.  Element by element against binary64, 2^-8 (|o| + A) + 2^-11 A with A = sum_j w_j |v_j| / l, and
the same bits in every run."""

import math
import random

import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu


def check(fm, dev, lens, H, H_kv, D, seed, runs=12):
    G, B, cu = H // H_kv, len(lens), [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    T, n_max = cu[-1], max(1, max(x for _, x in lens))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    q = wl.normal_bf16(seed, 150, (T, H, D), std=2.0).to(dev)
    k, v = (wl.normal_bf16(seed, 151 + i, (B, H_kv, n_max, D)).to(dev) for i in range(2))
    for b, (_, held) in enumerate(lens):
        k[b, :, held:], v[b, :, held:] = float("nan"), float("inf")
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device=dev)
    ws = torch.zeros(fm.fmlp_prefill_workspace_bytes(T, B, H, H_kv, D), dtype=torch.uint8, device=dev)
    args = (q, k, v, i32(cu), i32([x for _, x in lens]), 1 / math.sqrt(D), out, ws)
    fm.fmlp_attn_prefill(*args)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    for b, (new, held) in enumerate(lens):
        K, V = (t[b, :, :held].double().repeat_interleave(G, 0) for t in (k, v))
        rows = torch.arange(held - new, held, device=dev)
        x = q[cu[b]:cu[b + 1]].double().transpose(0, 1)
        z = (x @ K.mT / math.sqrt(D)).masked_fill(torch.arange(held, device=dev) > rows[:, None], -math.inf)
        w = torch.nan_to_num(torch.softmax(z, -1))
        o, a = w @ V, w @ V.abs()
        got = out[cu[b]:cu[b + 1]].double().transpose(0, 1)
        assert torch.all((got - o).abs() <= 2.0 ** -8 * (o.abs() + a) + 2.0 ** -11 * a), (b, lens[b])
    first = out.clone()
    for _ in range(runs):
        fm.fmlp_attn_prefill(*args)
        assert torch.equal(out, first)


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("G,H_kv", [(65, 3), (128, 2), (43, 4), (32, 8), (8, 8), (1, 8)])
def test_odd_numbers_of_tiles(cuda_device, G, H_kv, D):
    import token_phase_swiglu_b200 as fm
    rng = random.Random(G * D)
    tile = 128 // G
    lens = []
    for _ in range(24):                          # one, three, five tiles over a few units
        n = tile * rng.choice((0, 2, 4)) + rng.randint(1, tile)
        n = min(n, 300)
        lens.append((n, n + rng.choice((0, rng.randint(0, 600)))))
    check(fm, cuda_device, lens, G * H_kv, H_kv, D, seed=G + D)


@pytest.mark.parametrize("D", [64, 96, 128])
def test_many_short_segments(cuda_device, D):
    """One token a sequence beside longer ones: most segments have one tile only."""
    import token_phase_swiglu_b200 as fm
    rng = random.Random(D)
    lens = [(rng.choice((1, 1, 1, 2, 3, 5)), 0) for _ in range(400)]
    lens = [(n, n + rng.randint(0, 700)) for n, _ in lens]
    check(fm, cuda_device, lens, 64, 1, D, seed=D)
    check(fm, cuda_device, lens, 8, 8, D, seed=D + 1)
