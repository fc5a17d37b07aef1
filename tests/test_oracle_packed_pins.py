"""Pins of the packed-batch oracle (oracle/packed.py) on the CPU: against the single-token
oracle, closed forms, torch and scipy -- never against the CUDA path."""

import math

import numpy as np
import pytest
import scipy.special
import torch

import oracle
from oracle import packed

rng = np.random.default_rng(5)


def test_plain_frequencies_are_the_single_token_oracles():
    assert np.allclose(7.0 * packed.rope_frequencies(1e4, 64), oracle.rope_angles(7, 64, 1e4), rtol=1e-15)


@pytest.mark.parametrize("scaling", ["linear", "bands", "yarn"])
def test_scaled_frequencies_lie_between_the_plain_and_the_divided(scaling):
    plain = packed.rope_frequencies(5e5, 128)
    f = packed.rope_frequencies(5e5, 128, scaling, factor=8.0, low=1.0, high=32.0, original_ctx=8192)
    assert np.all(f <= plain * (1 + 1e-12)) and np.all(f >= plain / 8 * (1 - 1e-12))
    if scaling == "linear":
        assert np.allclose(f, plain / 8)
    else:  # fast pairs keep theirs, slow ones are divided, and the share never falls
        assert f[0] == plain[0] and math.isclose(f[-1], plain[-1] / 8, rel_tol=1e-12)
        assert np.all(np.diff(plain / f) >= -1e-12)


def test_bands_keep_and_divide_at_their_borders():
    ctx, low, high = 8192, 1.0, 4.0
    plain = packed.rope_frequencies(5e5, 128)
    f = packed.rope_frequencies(5e5, 128, "bands", factor=8.0, low=low, high=high, original_ctx=ctx)
    turns = ctx * plain / (2 * math.pi)
    assert np.all(f[turns >= high] == plain[turns >= high])
    assert np.allclose(f[turns < low], plain[turns < low] / 8, rtol=1e-15)


def test_half_rotation_is_the_single_token_oracles():
    x = rng.standard_normal((3, 96))
    assert np.allclose(packed.rotate(x, 41, packed.rope_frequencies(1e4, 96)), oracle.rope(x, 41, 1e4), atol=1e-14)


def test_adjacent_pairs_are_the_half_rotation_reordered():
    x = rng.standard_normal((2, 64))
    f = packed.rope_frequencies(1e4, 64)
    order = np.arange(64).reshape(2, 32).T.ravel()   # half-layout index of each adjacent position
    back = np.argsort(order)
    y = packed.rotate(x[:, order], 9, f, interleaved=True)
    assert np.allclose(y[:, back], packed.rotate(x, 9, f), atol=1e-14)


def test_partial_rotation_and_amplitude():
    x = rng.standard_normal((2, 96))
    y = packed.rotate(x, 5, packed.rope_frequencies(1e4, 48), amplitude=1.5)
    assert np.array_equal(y[:, 48:], x[:, 48:])
    assert np.allclose(np.linalg.norm(y[:, :48], axis=1), 1.5 * np.linalg.norm(x[:, :48], axis=1))


def test_head_norm_has_unit_mean_square():
    x = 100 * rng.standard_normal((4, 128))
    assert np.allclose(np.mean(packed.head_norm(x, np.ones(128), 0.0) ** 2, axis=1), 1.0)


def test_quantized_rows():
    x = rng.standard_normal((50, 64)) * np.exp(rng.standard_normal((50, 1)))
    q, s = packed.quantize_kv(x)
    assert np.all(np.abs(q * s[:, None].astype(np.float64) - x) <= 0.5 * s[:, None] * (1 + 1e-5))
    assert np.all(np.max(np.abs(q.astype(int)), axis=1) == 127)
    q, s = packed.quantize_kv(np.zeros((1, 64)))
    assert s[0] == 0 and not q.any()


def test_positions_of_ragged_and_padded_batches():
    assert packed.positions([1, 3, 3, 4], [5, 9, 1], 6) == [None, (0, 3), (0, 4), (2, 0), None, None]
    assert packed.positions([0, 3], [1], 3) == [None, None, (0, 0)]


def test_causal_attention_equals_torch_on_a_whole_prompt():
    n, H, H_kv, D = 9, 4, 2, 16
    q, K, V = rng.standard_normal((n, H, D)), rng.standard_normal((1, H_kv, n, D)), rng.standard_normal((1, H_kv, n, D))
    got = packed.causal_attention(q, K, V, [0, n], [n], 0.25)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), torch.from_numpy(K[0]).repeat_interleave(2, 0),
        torch.from_numpy(V[0]).repeat_interleave(2, 0), is_causal=True, scale=0.25).transpose(0, 1).numpy()
    assert np.allclose(got, want, atol=1e-13)


def test_causal_attention_of_one_token_is_the_decode_oracles():
    H, H_kv, D, n = 4, 2, 16, 12
    q, K, V = rng.standard_normal((1, H, D)), rng.standard_normal((1, H_kv, 20, D)), rng.standard_normal((1, H_kv, 20, D))
    got = packed.causal_attention(q, K, V, [0, 1], [n], 0.3)
    assert np.allclose(got[0], oracle.decode_attention(q[0], K[0, :, :n], V[0, :, :n], 0.3), atol=1e-14)


def test_tokens_without_rows_give_zeros_and_others_nothing():
    q = rng.standard_normal((5, 1, 8))
    K = V = rng.standard_normal((1, 1, 4, 8))
    out = packed.causal_attention(q, K, V, [1, 4], [2], 1.0)
    assert np.all(np.isnan(out[[0, 4]])) and np.all(out[1] == 0)
    assert np.allclose(out[2], V[0, 0, :1])


def test_int8_attention_equals_scipy():
    q = rng.standard_normal((2, 2, 8))
    kq, vq = (rng.integers(-127, 128, (2, 1, 6, 8)).astype(np.int8) for _ in range(2))
    ks, vs = (rng.random((2, 1, 6)).astype(np.float32) / 64 for _ in range(2))
    out = packed.decode_attention_q8(q, kq, ks, vq, vs, [4, 0], 0.5)
    K, V = kq[0, 0, :4] * ks[0, 0, :4, None].astype(float), vq[0, 0, :4] * vs[0, 0, :4, None].astype(float)
    assert np.allclose(out[0], scipy.special.softmax(0.5 * q[0] @ K.T, axis=1) @ V, atol=1e-13)
    assert np.all(out[1] == 0)
