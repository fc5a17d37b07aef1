"""The attention-side operators of a decoder layer, as cases to be measured.

Five calls that work on one packed batch of new tokens and its KV cache:

* ``rope``     fmlp_rope_append: per-head norms (optional) and rotation of q and k,
               the rotated keys and the values written to a bf16 cache;
* ``q8_write`` fmlp_rope_append_q8 and fmlp_kv_read_q8: the same into an int8 cache
               (one f32 scale a row), and the held rows read back as bf16;
* ``prefill``  fmlp_attn_prefill: causal attention of all new tokens over the cache;
* ``q8_decode`` fmlp_attn_decode_q8: attention of one token a sequence over the int8 cache.

A batch has B sequences with n_b new tokens each, packed one after another
(``cu`` [B + 1]), and ``kv_len`` [B] rows of cache held once the new tokens are
in it; token i of sequence b stands at position kv_len[b] - n_b + i.  Lengths
are a function of the case alone, values of the seed alone.

With ``own`` false, ``run`` computes the plain form in elementary torch
operations; with ``own`` true, it makes the library's calls.
"""

import math
import random

import torch

own = False

EPS = 1e-6

# Head shapes (query heads, KV heads, head dimension) of the attention steps
# this repository measures, then generic ones.
HEADS = ((32, 8, 128), (32, 32, 96), (4, 2, 64), (8, 1, 128), (16, 16, 64), (12, 4, 96), (40, 8, 128), (6, 2, 128))


def listed():
    return [
        # one decode step of 8 sequences, rotation scaled in bands for a long context
        dict(name="rope_decode_8", op="rope", B=8, n=1, even=True, ctx=4096, H=32, Hkv=8, D=128, rot=128,
             pairs="half", scaling="bands", norms=False, lens=1),
        # a ragged batch of prompts with per-head norms, adjacent pairs over half of the head
        dict(name="rope_norm_ragged", op="rope", B=5, n=701, even=False, ctx=997, H=12, Hkv=4, D=96, rot=48,
             pairs="adjacent", scaling="linear", norms=True, lens=2),
        # a long prompt, norms and rotation over the whole head
        dict(name="rope_norm_prompt_8192", op="rope", B=1, n=8192, even=True, ctx=8192, H=32, Hkv=8, D=128, rot=128,
             pairs="half", scaling="yarn", norms=True, lens=3),
        # a turn of 37 tokens on a short int8 cache, the cache read back for its prefill
        dict(name="q8_write_turn", op="q8_write", B=1, n=37, even=True, ctx=301, H=32, Hkv=8, D=128, rot=128,
             pairs="half", scaling="none", norms=False, lens=4),
        # four prompts written to an int8 cache and read back
        dict(name="q8_write_prompts", op="q8_write", B=4, n=2048, even=False, ctx=4096, H=32, Hkv=32, D=96, rot=96,
             pairs="half", scaling="none", norms=False, lens=5),
        # a verify batch: 32 sequences of 4 draft tokens over caches of up to 4k rows
        dict(name="prefill_verify_32x4", op="prefill", B=32, n=4, even=True, ctx=4096, H=32, Hkv=8, D=128, lens=6),
        # a 2048-token prompt
        dict(name="prefill_prompt_2048", op="prefill", B=1, n=2048, even=True, ctx=2048, H=32, Hkv=8, D=128, lens=7),
        # one KV head per query head, a 4k prompt
        dict(name="prefill_prompt_4096_d96", op="prefill", B=1, n=4096, even=True, ctx=4096, H=32, Hkv=32, D=96, lens=8),
        # ragged prompts, some of them continuing a held cache
        dict(name="prefill_packed_ragged", op="prefill", B=9, n=1531, even=False, ctx=2500, H=16, Hkv=4, D=64, lens=9),
        # the longest prompt
        dict(name="prefill_prompt_8192", op="prefill", B=1, n=8192, even=True, ctx=8192, H=32, Hkv=8, D=128, lens=10),
        # one sequence with a full 4k cache
        dict(name="q8_decode_1x4096", op="q8_decode", B=1, n=1, even=True, ctx=4096, H=32, Hkv=32, D=96, lens=11),
        # sixteen sequences of up to 16k rows
        dict(name="q8_decode_16x16384", op="q8_decode", B=16, n=1, even=False, ctx=16384, H=32, Hkv=8, D=128, lens=12),
    ]


def draw(rng):
    op = rng.choice(("rope", "q8_write", "prefill", "prefill", "q8_decode", "q8_decode"))
    H, Hkv, D = rng.choice(HEADS)
    log = lambda lo, hi: max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))  # noqa: E731
    case = dict(op=op, H=H, Hkv=Hkv, D=D, even=rng.random() < 0.3, lens=rng.randrange(1 << 30))
    if op == "q8_decode":
        B = log(1, 24)
        return dict(case, B=B, n=1, ctx=log(16, min(60000, 260000 // B)))
    if op == "prefill":
        if rng.random() < 0.3:  # a few tokens a sequence
            B = log(1, 40)
            return dict(case, B=B, n=rng.randint(1, 9), ctx=log(16, 120000 // B))
        n = log(3, min(8000, round(7000 * math.sqrt(4096 / (H * D)))))
        B = max(1, min(rng.randint(1, 12), 8000 // n, int(60e6 / (n * n)) or 1))
        return dict(case, B=B, n=n, ctx=min(8192, n + (log(1, 2000) if rng.random() < 0.5 else 0)))
    n = log(1, 6000)
    B = max(1, min(log(1, 16), 8000 // n))
    return dict(case, B=B, n=n, ctx=n + log(1, 2000), rot=rng.choice((D, D, D // 2)), pairs=rng.choice(("half", "adjacent")),
                scaling=rng.choice(("none", "linear", "bands", "yarn")), norms=rng.random() < 0.5)


def lengths(case):
    """[(new tokens, rows held after them)] of each sequence; the first one has the case's largest."""
    r = random.Random(case["lens"])
    got = [(case["n"], case["ctx"])]
    while len(got) < case["B"]:
        n = case["n"] if case["even"] or case["n"] < 2 else r.randint(1, case["n"])
        held = case["ctx"] - case["n"]
        got.append((n, n + (held if case["even"] or held < 1 else r.randint(0, held))))
    return got


def rotation(case):
    """The rotation's settings: base, scaling of the frequencies, amplitude of the cosines and sines."""
    s = dict(theta=500000.0, rotary_dim=case["rot"], interleaved=case["pairs"] == "adjacent", scaling=case["scaling"])
    if case["scaling"] == "linear":
        s.update(factor=4.0)
    if case["scaling"] == "bands":
        s.update(factor=8.0, low=1.0, high=4.0, original_ctx=2048)
    if case["scaling"] == "yarn":
        s.update(factor=4.0, low=1.0, high=32.0, original_ctx=2048, amplitude=0.1 * math.log(4.0) + 1.0)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    bf = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    lens = lengths(case)
    B, H, Hkv, D = case["B"], case["H"], case["Hkv"], case["D"]
    T, n_max = sum(n for n, _ in lens), max(held for _, held in lens)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    s = dict(op=case["op"], B=B, H=H, Hkv=Hkv, D=D, T=T, n_max=n_max, longest=max(n for n, _ in lens),
             cu=torch.tensor(cu, dtype=torch.int32, device=dev),
             kv_len=torch.tensor([held for _, held in lens], dtype=torch.int32, device=dev))
    if case["op"] in ("rope", "q8_write"):
        # q, k and v are column ranges of one projection's output
        qkv = bf(T, (H + 2 * Hkv) * D)
        q, k, v = qkv.split((H * D, Hkv * D, Hkv * D), dim=1)
        s.update(q=q.unflatten(1, (H, D)), k=k.unflatten(1, (Hkv, D)), v=v.unflatten(1, (Hkv, D)), rotation=rotation(case),
                 q_gamma=1 + bf(D, std=0.1) if case["norms"] else None,
                 k_gamma=1 + bf(D, std=0.1) if case["norms"] else None,
                 q_out=torch.empty(T, H, D, dtype=torch.bfloat16, device=dev))
    if case["op"] == "prefill":
        s.update(q=bf(T, H, D, std=2.0), out=torch.empty(T, H, D, dtype=torch.bfloat16, device=dev))
    if case["op"] in ("rope", "prefill"):
        s.update(k_cache=bf(B, Hkv, n_max, D), v_cache=bf(B, Hkv, n_max, D))
    if case["op"] in ("q8_write", "q8_decode"):
        for c in ("k", "v"):
            x = torch.randn(B, Hkv, n_max, D, generator=g, device=dev)
            x = x * torch.exp(0.3 * torch.randn(B, Hkv, n_max, 1, generator=g, device=dev))
            s[c + "_s"] = x.abs().amax(-1) / 127
            s[c + "_q"] = torch.round(x / s[c + "_s"][..., None]).to(torch.int8)
    if case["op"] == "q8_write":
        s.update(k_cache=torch.zeros(B, Hkv, n_max, D, dtype=torch.bfloat16, device=dev),
                 v_cache=torch.zeros(B, Hkv, n_max, D, dtype=torch.bfloat16, device=dev))
    if case["op"] == "q8_decode":
        s.update(q=bf(B, H, D, std=2.0), out=torch.empty(B, H, D, device=dev))
    s["scale"] = 1.0 / math.sqrt(D)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def tokens(s):
    """Sequence and position of every packed token."""
    t = torch.arange(s["T"], device=s["cu"].device)
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return b, s["kv_len"].long()[b] - s["cu"].long()[b + 1] + t


def frequencies(r, dev):
    R, base = r["rotary_dim"], r["theta"]
    i = torch.arange(R // 2, dtype=torch.float64, device=dev)
    f = base ** (-2.0 * i / R)
    if r["scaling"] == "linear":
        f = f / r["factor"]
    if r["scaling"] == "bands":
        turns = r["original_ctx"] * f / (2 * math.pi)
        keep = ((turns - r["low"]) / (r["high"] - r["low"])).clamp(0, 1)
        f = keep * f + (1 - keep) * f / r["factor"]
    if r["scaling"] == "yarn":
        at = lambda turns: R * math.log(r["original_ctx"] / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(r["high"])), 0), min(math.ceil(at(r["low"])), R - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = ramp * f / r["factor"] + (1 - ramp) * f
    return f


def normed(x, gamma):
    x = x.float()
    return x if gamma is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()


def rotated(x, pos, r):
    R = r["rotary_dim"]
    a = pos.double()[:, None] * frequencies(r, x.device)
    c, s = ((f(a) * r.get("amplitude", 1.0)).float()[:, None] for f in (torch.cos, torch.sin))
    y = x.clone()
    lo, hi = (slice(0, R, 2), slice(1, R, 2)) if r["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., lo] * s + x[..., hi] * c
    return y


def quantized(x):
    s = x.abs().amax(-1) / 127
    return torch.where(s[..., None] > 0, torch.round(x / s[..., None]), 0).clamp(-127, 127).to(torch.int8), s


def plain_rope(s):
    b, pos = tokens(s)
    q = rotated(normed(s["q"], s["q_gamma"]), pos, s["rotation"]).to(torch.bfloat16)
    k = rotated(normed(s["k"], s["k_gamma"]), pos, s["rotation"])
    if s["op"] == "rope":
        s["k_cache"][b, :, pos] = k.to(torch.bfloat16)
        s["v_cache"][b, :, pos] = s["v"]
    else:
        s["k_q"][b, :, pos], s["k_s"][b, :, pos] = quantized(k)
        s["v_q"][b, :, pos], s["v_s"][b, :, pos] = quantized(s["v"].float())
        held = (torch.arange(s["n_max"], device=b.device) < s["kv_len"][:, None])[:, None, :, None]
        s["k_cache"].copy_(torch.where(held, s["k_q"] * s["k_s"][..., None], s["k_cache"]))
        s["v_cache"].copy_(torch.where(held, s["v_q"] * s["v_s"][..., None], s["v_cache"]))
    return q, s["k_cache"], s["v_cache"]


def plain_prefill(s):
    b, pos = tokens(s)
    B, H, Hkv, D, n = s["B"], s["H"], s["Hkv"], s["D"], s["longest"]
    at = torch.arange(s["T"], device=b.device) - s["cu"].long()[b]
    q = torch.zeros(B, n, H, D, device=b.device)
    q[b, at] = s["q"].float() * s["scale"]
    last = torch.full((B, n), -1, device=b.device)
    last[b, at] = pos
    q = q.view(B, n, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    p = (q @ s["k_cache"].float().mT).view(B, H, n, -1)
    p.masked_fill_(torch.arange(s["n_max"], device=b.device) > last[:, None, :, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1)
    o = (p.view(B, Hkv, -1, s["n_max"]) @ s["v_cache"].float()).view(B, H, n, D) / total[..., None]
    return o.transpose(1, 2)[b, at].to(torch.bfloat16)


def plain_q8_decode(s):
    B, H, Hkv, D = s["B"], s["H"], s["Hkv"], s["D"]
    q = s["q"].float().view(B, Hkv, H // Hkv, D) * s["scale"]
    p = q @ (s["k_q"] * s["k_s"][..., None]).mT
    p.masked_fill_((torch.arange(s["n_max"], device=q.device) >= s["kv_len"][:, None])[:, None, None], -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp()
    o = p @ (s["v_q"] * s["v_s"][..., None])
    return (o / p.sum(-1, keepdim=True)).view(B, H, D)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def workspace(s, need):
    """Zero-filled once, kept with the program's other buffers."""
    if "workspace" not in s:
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device=s["cu"].device)
    return s["workspace"]


def own_calls(s):
    import token_phase_swiglu_b200 as fm
    if s["op"] in ("rope", "q8_write"):
        if "rope" not in s:
            s["rope"] = fm.FmlpRope(**s["rotation"])
        ws = workspace(s, fm.CONTROL_BYTES)
        if s["op"] == "rope":
            fm.fmlp_rope_append(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], s["rope"], s["q_out"], s["k_cache"],
                                s["v_cache"], ws, q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=EPS)
        else:
            fm.fmlp_rope_append_q8(s["q"], s["k"], s["v"], s["cu"], s["kv_len"], s["rope"], s["q_out"], s["k_q"],
                                   s["k_s"], s["v_q"], s["v_s"], ws, q_gamma=s["q_gamma"], k_gamma=s["k_gamma"],
                                   eps=EPS)
            fm.fmlp_kv_read_q8(s["k_q"], s["k_s"], s["v_q"], s["v_s"], s["kv_len"], s["k_cache"], s["v_cache"], ws)
        return s["q_out"], s["k_cache"], s["v_cache"]
    if s["op"] == "prefill":
        ws = workspace(s, fm.fmlp_prefill_workspace_bytes(s["T"], s["B"], s["H"], s["Hkv"], s["D"]))
        fm.fmlp_attn_prefill(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["kv_len"], s["scale"], s["out"], ws)
        return s["out"]
    ws = workspace(s, fm.fmlp_attn_q8_workspace_bytes(s["B"], s["H"], s["Hkv"], s["D"]))
    fm.fmlp_attn_decode_q8(s["q"], s["k_q"], s["k_s"], s["v_q"], s["v_s"], s["kv_len"], s["scale"], s["out"], ws)
    return s["out"]


def run(state):
    if own:
        return own_calls(state)
    return {"rope": plain_rope, "q8_write": plain_rope, "prefill": plain_prefill,
            "q8_decode": plain_q8_decode}[state["op"]](state)


def work(case):
    lens = lengths(case)
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    T, rows = sum(n for n, _ in lens), sum(held for _, held in lens)
    row8 = D + 4  # an int8 row and its scale
    if case["op"] == "rope":
        return {"bytes": 2 * 2 * T * (H + 2 * Hkv) * D, "flops": 3 * T * (H + Hkv) * D}
    if case["op"] == "q8_write":
        wrote = 2 * T * (2 * H + 2 * Hkv) * D + 2 * T * Hkv * row8
        return {"bytes": wrote + 2 * rows * Hkv * (row8 + 2 * D), "flops": 3 * T * (H + Hkv) * D + 4 * T * Hkv * D}
    if case["op"] == "prefill":
        pairs = sum(n * (held - n) + n * (n + 1) // 2 for n, held in lens)
        return {"bytes": 2 * 2 * T * H * D + 2 * 2 * rows * Hkv * D, "flops": 4 * D * H * pairs}
    return {"bytes": 2 * rows * Hkv * row8 + case["B"] * H * D * (2 + 4), "flops": 4 * D * H * rows}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    lens, H, Hkv, D = lengths(case), case["H"], case["Hkv"], case["D"]
    start = [0]
    for n, _ in lens:
        start.append(start[-1] + n)
    if case["op"] == "prefill":
        out = torch.empty(s["T"], H, D, dtype=torch.float64, device="cuda")
        for b, (n, held) in enumerate(lens):
            free = torch.ones(n, held, dtype=torch.bool, device="cuda").tril(held - n)
            for h in range(H):
                K, V = (s[c][b, h // (H // Hkv), :held].double() for c in ("k_cache", "v_cache"))
                z = s["q"][start[b]:start[b + 1], h].double() @ K.T / math.sqrt(D)
                out[start[b]:start[b + 1], h] = torch.softmax(torch.where(free, z, -math.inf), -1) @ V
        return out
    if case["op"] == "q8_decode":
        out = torch.empty(len(lens), H, D, dtype=torch.float64, device="cuda")
        for b, (_, held) in enumerate(lens):
            K, V = (s[c + "_q"][b, :, :held].double() * s[c + "_s"][b, :, :held, None].double() for c in ("k", "v"))
            z = torch.einsum("gid,gjd->gij", s["q"][b].double().view(Hkv, H // Hkv, D), K) / math.sqrt(D)
            out[b] = torch.einsum("gij,gjd->gid", torch.softmax(z, -1), V).reshape(H, D)
        return out
    r, R = s["rotation"], case["rot"]
    f = []
    for i in range(R // 2):
        w = r["theta"] ** (-2.0 * i / R)
        if r["scaling"] == "linear":
            w /= r["factor"]
        if r["scaling"] == "bands":
            wave = 2 * math.pi / w
            if wave > r["original_ctx"] / r["low"]:
                w /= r["factor"]
            elif wave > r["original_ctx"] / r["high"]:
                mix = (r["original_ctx"] / wave - r["low"]) / (r["high"] - r["low"])
                w = (1 - mix) * w / r["factor"] + mix * w
        if r["scaling"] == "yarn":
            edge = [R / 2 * math.log(r["original_ctx"] / (2 * math.pi * t), r["theta"]) for t in (r["high"], r["low"])]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), R - 1)
            mix = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            w = mix * w / r["factor"] + (1 - mix) * w
        f.append(w)
    f = torch.tensor(f, dtype=torch.float64, device="cuda")

    def turn(x, gamma, pos):
        x = x.double()
        if gamma is not None:
            x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * gamma.double()
        z = x[..., :R].unflatten(-1, (R // 2, 2)) if r["interleaved"] else x[..., :R].unflatten(-1, (2, R // 2)).mT
        z = torch.view_as_complex(z.contiguous())
        z = torch.view_as_real(z * torch.polar(torch.full_like(f, r.get("amplitude", 1.0)), pos[:, None] * f)[:, None])
        return torch.cat([(z if r["interleaved"] else z.mT).flatten(-2), x[..., R:]], -1)

    if case["op"] == "rope":
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    else:
        k_cache, v_cache = torch.zeros_like(s["k_cache"], dtype=torch.float64), torch.zeros_like(s["v_cache"], dtype=torch.float64)
    q = torch.empty(s["T"], H, D, dtype=torch.float64, device="cuda")
    for b, (n, held) in enumerate(lens):
        at = slice(start[b], start[b + 1])
        pos = torch.arange(held - n, held, dtype=torch.float64, device="cuda")
        q[at] = turn(s["q"][at], s["q_gamma"], pos)
        new = {"k": turn(s["k"][at], s["k_gamma"], pos), "v": s["v"][at].double()}
        for c, cache in (("k", k_cache), ("v", v_cache)):
            x = new[c]
            if case["op"] == "q8_write":
                step = (x.abs().amax(-1, keepdim=True) / 127).float().double()
                x = torch.round(x / step).clamp(-127, 127) * step
                cache[b, :, :held - n] = s[c + "_q"][b, :, :held - n].double() * s[c + "_s"][b, :, :held - n, None].double()
            cache[b, :, held - n:held] = x.transpose(0, 1)
    return q, k_cache, v_cache
