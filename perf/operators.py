"""The operators of a cross-attention site, as they are measured.

Three operators that run one after the other where a block of a transformer
(a diffusion transformer's latent tokens, or one new token of a decoder)
attends to the states of an encoder:

  norm       add_rms_norm_quant: the residual's addition, the root-mean-square
             norm and the E4M3 codes that the next linear layer reads, with a
             static scale or with one scale for each token;
  linear     fp8_linear_w8a8_pertoken(_group): the E4M3 linear layer with a
             scale for each token and one for each output channel;
  attention  cross_attention: softmax attention of the queries over the
             encoder's keys and values, of another length, with lengths or a
             mask for each sample and shared key/value heads, written in
             16 bits or as E4M3 codes with a static scale.

`run` computes them in elementary operations in 32 bits where `own` is false,
and through the package's entry points where it is true.  Codes are returned
as the E4M3 values that they are.  `exact` gives the same outputs from the
definition in 64 bits; in the place of E4M3 values it has the values that
they round.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
TINY = 2.0 ** -126      # smallest normal binary32: the least scale of a token


def listed():
    return [
        # one new token of a decoder: the norm before its next projection
        dict(name="norm_token", op="norm", rows=1, width=4096, dtype="bf16", static=False, residual=True),
        # a ragged prompt, a width that is no power of two, a calibrated scale
        dict(name="norm_prompt", op="norm", rows=333, width=2312, dtype="f16", static=True, residual=True),
        # the latent tokens of a diffusion transformer (13 x 30 x 53 of them)
        dict(name="norm_latent", op="norm", rows=20670, width=4096, dtype="bf16", static=False, residual=True),
        # the query projection of one new token
        dict(name="linear_token", op="linear", rows=1, inner=4096, outs=4096, group=1),
        # a batch of new tokens through the widest layer (the down projection)
        dict(name="linear_batch_down", op="linear", rows=16, inner=16384, outs=4096, group=1),
        # keys and values of a prompt's encoder states, with shared heads
        dict(name="linear_prompt_kv", op="linear", rows=333, inner=4096, outs=1024, group=2),
        # the query projection of all latent tokens
        dict(name="linear_latent", op="linear", rows=20670, inner=4096, outs=4096, group=1),
        # one new token over a short prompt: the smallest call, where latency counts
        dict(name="attn_token_prompt", op="attention", batch=1, queries=1, keys=512, heads=32, kv_heads=32, dim=128,
             dtype="bf16", lens=False, mask=False, codes=False),
        # a batch of new tokens over long encoder states with lengths of their own, shared heads
        dict(name="attn_token_long", op="attention", batch=8, queries=1, keys=20670, heads=32, kv_heads=8, dim=128,
             dtype="bf16", lens=True, mask=False, codes=False),
        # small heads, a mask over the prompt, odd lengths
        dict(name="attn_mask", op="attention", batch=3, queries=1077, keys=999, heads=20, kv_heads=4, dim=64,
             dtype="f16", lens=False, mask=True, codes=False),
        # latent tokens over a padded prompt, written as codes for the out-projection
        dict(name="attn_latent_prompt", op="attention", batch=2, queries=20670, keys=512, heads=32, kv_heads=32,
             dim=128, dtype="bf16", lens=True, mask=False, codes=True),
        # a block of tokens over the states of all latent tokens: the largest product
        dict(name="attn_block_latent", op="attention", batch=1, queries=4096, keys=20670, heads=32, kv_heads=8,
             dim=128, dtype="bf16", lens=False, mask=False, codes=False),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "linear", "attention", "attention"])
    if op == "norm":
        return dict(op=op, rows=_spread(rng, 1, 20670), width=_spread(rng, 64, 16384, 8), dtype=rng.choice(["bf16", "f16"]),
                    static=rng.random() < 0.5, residual=rng.random() < 0.8)
    if op == "linear":
        c = dict(op=op, rows=_spread(rng, 1, 20670), inner=_spread(rng, 256, 16384, 16), outs=_spread(rng, 256, 16384, 16),
                 group=rng.choice([1, 1, 2, 3]))
        while c["rows"] * c["inner"] * c["outs"] * c["group"] > 20670 * 4096 * 4096:
            c["rows"] = (c["rows"] + 1) // 2
        return c
    kv = rng.choice([1, 2, 4, 8, 16])
    c = dict(op=op, batch=rng.choice([1, 1, 2, 3, 5, 8]), queries=_spread(rng, 1, 20670), keys=_spread(rng, 1, 20670),
             heads=kv * rng.choice([1, 1, 2, 3, 4, 7, 8]), kv_heads=kv, dim=rng.choice([64, 64, 80, 96, 128, 128]),
             dtype=rng.choice(["bf16", "f16"]), lens=rng.random() < 0.4, mask=rng.random() < 0.3, codes=rng.random() < 0.3)
    if rng.random() < 0.3:
        c["queries"] = 1
    while c["batch"] * c["heads"] * c["queries"] * c["keys"] > 32 * 4096 * 20670:
        side = "queries" if c["queries"] > 1 else "keys"
        c[side] = (c[side] + 1) // 2
    return c


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)

    def normal(shape, std, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def codes_of(v, scale):
        return (v / scale).clamp(-448.0, 448.0).to(F8).view(torch.uint8)

    u8 = dict(dtype=torch.uint8, device="cuda")
    if case["op"] == "norm":
        M, K, dt = case["rows"], case["width"], TYPES[case["dtype"]]
        s["x"] = normal((M, K), 0.5, dt)
        s["residual"] = normal((M, K), 1.0, dt) if case["residual"] else None
        if s["residual"] is not None:                       # some heavy channels, as hidden states have
            s["residual"][:, :: max(K // 7, 1)] *= 8
        s["weight"] = (1.0 + normal((K,), 0.1)).to(dt)
        s["s_in"] = torch.full((1,), 8.0 / 448.0, device="cuda") if case["static"] else None
        s["q"] = torch.empty((M, K), **u8)
        s["s_tok"] = None if case["static"] else torch.empty((M,), device="cuda")
        s["res_out"] = torch.empty((M, K), dtype=dt, device="cuda") if case["residual"] else None
    elif case["op"] == "linear":
        M, K, N, G = case["rows"], case["inner"], case["outs"], case["group"]
        x = normal((M, K), 1.0)
        s["s_tok"] = (x.abs().amax(1) / 448.0).clamp_min(TINY)
        s["x"] = codes_of(x, s["s_tok"][:, None])
        s["w"], s["s_ch"] = [], []
        for i in range(G):
            w = normal((N, K), 0.02) * (0.5 + torch.rand((N, 1), generator=g, device="cuda"))
            c = w.abs().amax(1) / 448.0
            s["w"].append(codes_of(w, c[:, None]))
            s["s_ch"].append(c)
        s["y"] = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(G)]
    else:
        B, L, T, H, Hk, D = (case[k] for k in ("batch", "queries", "keys", "heads", "kv_heads", "dim"))
        dt = TYPES[case["dtype"]]
        s["q"] = normal((B, L, H, D), 1.0, dt)
        s["k"] = normal((B, T, Hk, D), 1.0, dt)
        s["v"] = normal((B, T, Hk, D), 1.0, dt)
        s["kv_len"] = s["kv_mask"] = s["s_out"] = None
        if case["lens"]:                                     # between a half and all of the keys
            n = torch.randint((T + 1) // 2, T + 1, (B,), generator=g, device="cuda")
            s["kv_len"] = n.to(torch.int32)
        if case["mask"]:                                     # one key in five is padding
            s["kv_mask"] = torch.rand((B, T), generator=g, device="cuda") >= 0.2
        if case["codes"]:
            s["s_out"] = torch.full((1,), 3.0 / 448.0, device="cuda")
            s["out"] = torch.empty((B, L, H, D), **u8)
        else:
            s["out"] = torch.empty((B, L, H, D), dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"norm": _plain_norm, "linear": _plain_linear, "attention": _plain_attention}[s["op"]](s)


def _run_own(s):
    import w8a16_linear_gb300 as W
    if s["op"] == "norm":
        q, s_tok, res = W.add_rms_norm_quant(s["x"], s["residual"], s["weight"], eps=EPS, s_in=s["s_in"], out=s["q"],
                                             s_tok=s["s_tok"], res_out=s["res_out"])
        return {"q": q.view(F8), "s_tok": s_tok, "res": res}
    if s["op"] == "linear":
        if s["group"] == 1:
            return [W.fp8_linear_w8a8_pertoken(s["x"], s["s_tok"], s["w"][0], s["s_ch"][0], out=s["y"][0])]
        return W.fp8_linear_w8a8_pertoken_group(s["x"], s["s_tok"], s["w"], s["s_ch"], outs=s["y"])
    out = W.cross_attention(s["q"], s["k"], s["v"], kv_len=s["kv_len"], kv_mask=s["kv_mask"], s_out=s["s_out"],
                            out=s["out"])
    return out.view(F8) if s["codes"] else out


def _plain_norm(s):
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    h = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["weight"].float()
    if s["static"]:
        scale, s_tok = s["s_in"], None
    else:
        scale = (h.abs().amax(1, keepdim=True) / 448.0).clamp_min(TINY)
        s_tok = scale[:, 0]
    q = (h / scale).clamp(-448.0, 448.0).to(F8)
    return {"q": q, "s_tok": s_tok, "res": r.to(s["x"].dtype) if s["residual"] is not None else None}


def _plain_linear(s):
    x = s["x"].view(F8).float()
    return [((x @ w.view(F8).float().T) * s["s_tok"][:, None] * c).to(torch.bfloat16) for w, c in zip(s["w"], s["s_ch"])]


def _allowed(s):
    """[B, 1, 1, keys] truth values of the keys that count, or None for all."""
    T, ok = s["keys"], None
    if s["kv_len"] is not None:
        ok = torch.arange(T, device="cuda")[None, :] < s["kv_len"][:, None]
    if s["kv_mask"] is not None:
        ok = s["kv_mask"] if ok is None else ok & s["kv_mask"]
    return None if ok is None else ok[:, None, None, :]


def _plain_attention(s):
    B, L, T, H, Hk, D = (s[k] for k in ("batch", "queries", "keys", "heads", "kv_heads", "dim"))
    G = H // Hk
    # the query heads that share a key head stand one below the other
    q = s["q"].float().view(B, L, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, L * G, D)
    k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    p = q @ (k * D ** -0.5).transpose(2, 3)
    ok = _allowed(s)
    if ok is not None:
        p = p.masked_fill(~ok, float("-inf"))
        p = p.sub_(p.amax(3, keepdim=True).clamp_min(-1e38)).exp_()
        v = v.masked_fill(~ok.transpose(2, 3), 0.0)
    else:
        p = p.sub_(p.amax(3, keepdim=True)).exp_()
    n = p.sum(3, keepdim=True)
    o = torch.where(n > 0, (p @ v) / n, 0.0)
    o = o.view(B, Hk, L, G, D).permute(0, 2, 1, 3, 4).reshape(B, L, H, D)
    if s["codes"]:
        return (o / s["s_out"]).clamp(-448.0, 448.0).to(F8)
    return o.to(s["q"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "norm":
        M, K = case["rows"], case["width"]
        per = 2 + 1 + (4 if case["residual"] else 0)         # x, codes, residual in and out
        return {"bytes": M * K * per + 2 * K + 4 * (1 if case["static"] else M), "flops": 5 * M * K}
    if case["op"] == "linear":
        M, K, N, G = case["rows"], case["inner"], case["outs"], case["group"]
        return {"bytes": M * K + 4 * M + G * (N * K + 4 * N + 2 * M * N), "flops": 2 * M * N * K * G}
    B, L, T, H, Hk, D = (case[k] for k in ("batch", "queries", "keys", "heads", "kv_heads", "dim"))
    part = 1.0                                               # the keys that count, on average
    if case["lens"]:
        part *= 0.75
    if case["mask"]:
        part *= 0.8
    n = B * L * H * D * (2 + (1 if case["codes"] else 2)) + 2 * 2 * B * Hk * T * D * part
    n += (4 * B if case["lens"] else 0) + (B * T if case["mask"] else 0)
    return {"bytes": n, "flops": 4 * B * H * L * T * D * part}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        t = s["x"].double()
        if case["residual"]:
            t += s["residual"].double()
        res = t.clone() if case["residual"] else None
        power = torch.linalg.vector_norm(t, dim=1).square() / case["width"]
        t *= s["weight"].double()
        t /= (power + EPS).sqrt()[:, None]
        if case["static"]:
            return {"q": (t / s["s_in"].double()).clamp(-448, 448), "s_tok": None, "res": res}
        m = torch.maximum(t.amax(1), -t.amin(1)) / 448
        m = m.clamp_min(TINY)
        return {"q": t / m[:, None], "s_tok": m, "res": res}
    if case["op"] == "linear":
        a = s["x"].view(F8).double() * s["s_tok"].double()[:, None]
        return [torch.einsum("mk,nk->mn", a, w.view(F8).double() * c.double()[:, None]) for w, c in zip(s["w"], s["s_ch"])]
    B, L, H, D = s["q"].shape
    G = H // case["kv_heads"]
    out = torch.zeros((B, L, H, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        keep = torch.ones(case["keys"], dtype=torch.bool, device="cuda")
        if case["lens"]:
            keep[int(s["kv_len"][b]):] = False
        if case["mask"]:
            keep &= s["kv_mask"][b]
        at = keep.nonzero()[:, 0]
        if not len(at):
            continue
        for h in range(H):
            k, v = s["k"][b, at, h // G].double(), s["v"][b, at, h // G].double()
            for i in range(0, L, 8192):
                e = torch.softmax(s["q"][b, i:i + 8192, h].double() @ k.T / math.sqrt(D), dim=1)
                out[b, i:i + 8192, h] = e @ v
    return (out / s["s_out"].double()).clamp(-448, 448) if case["codes"] else out
