"""fp64 oracle of the calls on packed batches -- TEST INFRASTRUCTURE ONLY.

Plain restatements of what the pages' token-phase attention needs around it:
the norm and rotation of a prompt's queries and keys, the append of keys and
values to the cache (bf16, or int8 with one scale a row), the causal attention
of a packed batch over the cache, and the attention of one token a sequence
over an int8 cache.  The pages (FastTPS, section 三, components 1-2) give the
single-token step and the cache addressing only; the formats and scalings are
the library's own, as its header states them.
"""

from __future__ import annotations

import math

import numpy as np


def rope_frequencies(theta, R, scaling="none", factor=1.0, low=1.0, high=4.0, original_ctx=1):
    """The R/2 pair frequencies."""
    out = []
    for i in range(R // 2):
        w = theta ** (-2.0 * i / R)
        if scaling == "linear":
            w = w / factor
        elif scaling == "bands":
            turns = original_ctx * w / (2 * math.pi)
            if turns < low:
                w = w / factor
            elif turns < high:
                m = (turns - low) / (high - low)
                w = m * w + (1 - m) * w / factor
        elif scaling == "yarn":
            pair = lambda n: R * math.log(original_ctx / (2 * math.pi * n)) / (2 * math.log(theta))  # noqa: E731
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), R - 1)
            r = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            w = r * w / factor + (1 - r) * w
        out.append(w)
    return np.array(out)


def head_norm(x, gamma, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * gamma


def rotate(x, pos, freq, interleaved=False, amplitude=1.0):
    """x [..., D] with its first 2 len(freq) values rotated by pos * freq."""
    x = np.array(x, dtype=np.float64)
    n = len(freq)
    lo = [2 * i if interleaved else i for i in range(n)]
    hi = [2 * i + 1 if interleaved else i + n for i in range(n)]
    a = float(pos) * np.asarray(freq)
    c, s = amplitude * np.cos(a), amplitude * np.sin(a)
    x0, x1 = x[..., lo].copy(), x[..., hi].copy()
    x[..., lo] = x0 * c - x1 * s
    x[..., hi] = x0 * s + x1 * c
    return x


def quantize_kv(x):
    """int8 codes and binary32 scales of rows x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    s = (np.max(np.abs(x), axis=-1) / 127).astype(np.float32)
    s = np.where(s < 2.0 ** -125, np.float32(0), s)
    safe = np.where(s > 0, s, 1).astype(np.float64)
    q = np.where(s[..., None] > 0, np.clip(np.rint(x / safe[..., None]), -127, 127), 0)
    return q.astype(np.int8), s


def positions(cu, kv_len, T):
    """[(sequence, position)] of every token; None where it is in no sequence, or padding."""
    out = [None] * T
    for b in range(len(kv_len)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            p = kv_len[b] - n + i
            if p >= 0:
                out[cu[b] + i] = (b, p)
    return out


def causal_attention(q, K, V, cu, kv_len, scale):
    """o [T, H, D] of rotated queries q [T, H, D] over caches K, V [B, H_kv, n_max, D]; rows of
    tokens outside every sequence are NaN, padding tokens (no position) give zeros."""
    T, H, D = q.shape
    group = H // K.shape[1]
    out = np.full((T, H, D), np.nan)
    at = positions(cu, kv_len, T)
    for t in range(cu[0], cu[-1]):
        if at[t] is None:
            out[t] = 0.0
            continue
        b, p = at[t]
        for h in range(H):
            g = h // group
            z = scale * (K[b, g, : p + 1] @ q[t, h])
            w = np.exp(z - np.max(z))
            out[t, h] = (w / np.sum(w)) @ V[b, g, : p + 1]
    return out


def decode_attention_q8(q, k_q, k_s, v_q, v_s, kv_len, scale):
    """o [B, H, D] of q [B, H, D] over rows 0 .. kv_len[b] - 1 of an int8 cache (zeros if none)."""
    B, H, D = q.shape
    group = H // k_q.shape[1]
    out = np.zeros((B, H, D))
    for b in range(B):
        n = int(kv_len[b])
        for h in range(H if n else 0):
            g = h // group
            K = k_q[b, g, :n].astype(np.float64) * k_s[b, g, :n, None].astype(np.float64)
            V = v_q[b, g, :n].astype(np.float64) * v_s[b, g, :n, None].astype(np.float64)
            z = scale * (K @ q[b, h])
            w = np.exp(z - np.max(z))
            out[b, h] = (w / np.sum(w)) @ V
    return out
