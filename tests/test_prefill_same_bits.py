"""fmlp_attn_prefill gives the same bits whatever ran on the GPU before it and whatever stands beside a
sequence in the batch's memory: query rows of no token (128 is not a multiple of the heads a KV head,
or a sequence ends inside a tile) take no part in the others' results."""

import math

import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fm(cuda_device):
    import token_phase_swiglu_b200 as fm
    return fm


def attend(fm, q, k, v, cu, kv_len):
    dev = q.device
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    T, H, D = q.shape
    B, H_kv = k.shape[:2]
    out = torch.full_like(q, 7.0)
    ws = torch.zeros(fm.fmlp_prefill_workspace_bytes(T, B, H, H_kv, D), dtype=torch.uint8, device=dev)
    fm.fmlp_attn_prefill(q, k, v, i32(cu), i32(kv_len), 1 / math.sqrt(D), out, ws)
    assert fm.fmlp_device_status(ws) == fm.FMLP_OK
    return out


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("G", [3, 5, 6, 7, 12, 100])
def test_after_other_calls(fm, cuda_device, G, D):
    n, held = 3 * (128 // G) + 5, 2000
    q = wl.normal_bf16(G, 130, (n, G, D), std=2.0).to(cuda_device)
    k, v = (wl.normal_bf16(G, 131 + i, (1, 1, held, D)).to(cuda_device) for i in range(2))
    k = (k.float() * torch.linspace(0.2, 3, held, device=cuda_device)[:, None]).to(torch.bfloat16)
    # a call of whole tiles on every SM, its queries of other sizes: what it leaves in shared memory
    oq = wl.normal_bf16(G, 133, (2048, 16, D)).to(cuda_device)
    ok, ov = (wl.normal_bf16(G, 134 + i, (1, 16, 2048, D)).to(cuda_device) for i in range(2))
    want = None
    for size in (1.0, 100.0, 1e4, 0.0, float("inf"), float("nan"), 3.0):
        x = (oq.float() * size).to(torch.bfloat16)
        attend(fm, x, ok, ov, [0, 2048], [2048])
        got = attend(fm, q, k, v, [0, n], [held])
        want = got if want is None else want
        assert torch.all(torch.isfinite(got)) and torch.equal(got, want), size


@pytest.mark.parametrize("G,D", [(1, 64), (4, 128), (3, 96), (8, 64)])
def test_whatever_follows_in_the_batch(fm, cuda_device, G, D):
    """The tokens behind a sequence's last one, of no sequence here, with queries of any size."""
    n, T, held = 128 // G + 3, 128 // G * 4, 1500
    q = wl.normal_bf16(G, 140, (T, G, D), std=2.0).to(cuda_device)
    k, v = (wl.normal_bf16(G, 141 + i, (1, 1, held, D)).to(cuda_device) for i in range(2))
    k = (k.float() * torch.linspace(0.2, 3, held, device=cuda_device)[:, None]).to(torch.bfloat16)
    want = attend(fm, q, k, v, [0, n], [held])
    for size in (50.0, 0.0, float("inf"), float("nan")):
        q[n:] *= size
        got = attend(fm, q, k, v, [0, n], [held])
        assert torch.equal(got[:n], want[:n]), size
        assert torch.all(got[n:] == 7)
        q[n:] = 1.0
