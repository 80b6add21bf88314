"""The operators of a self-attention site over a paged cache, as they are measured.

Three operators that run one after the other where a decoder's block (or a
block of latent tokens that also looks back) attends to its own past:

  rope       qk_norm_rope: the root-mean-square norm of every head of the
             queries and keys and their rotation by position, in one pass;
  append     paged_kv_append: the same on the way into a paged cache of keys
             and values (16 bits, or E4M3 codes with static scales), for the
             new tokens of several sequences;
  attention  paged_attention: the new tokens of each sequence (one, or a chunk)
             over all of its cached positions, causal or not, written in
             16 bits or as E4M3 codes with a static scale.

`run` computes them in elementary operations in 32 bits (angles in 64) where
`own` is false, and through the package's entry points where it is true.  Codes
are returned as the E4M3 values that they are.  `exact` gives the same outputs
from the definition in 64 bits; in the place of E4M3 values it has the values
that they round.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
K_SCALE, V_SCALE, OUT_SCALE = 0.03125, 0.0234375, 0.0078125


def listed():
    return [
        # queries and keys of one new token: the smallest call, where latency counts
        dict(name="rope_token", op="rope", rows=1, heads=32, kv_heads=8, dim=128, rot=128, axes=1, interleaved=False,
             norm=True, amplitude=1.0, far=0, dtype="bf16"),
        # a ragged prompt, heads of a size that is no power of two, a part of each rotated, positions of a long context
        dict(name="rope_prompt", op="rope", rows=333, heads=20, kv_heads=4, dim=80, rot=32, axes=1, interleaved=True,
             norm=False, amplitude=1.125, far=1000000, dtype="f16"),
        # the latent tokens of a diffusion transformer (13 x 30 x 53 of them), rotated by frame, row and column
        dict(name="rope_latent", op="rope", rows=20670, heads=32, kv_heads=8, dim=128, rot=128, axes=3,
             interleaved=False, norm=True, amplitude=1.0, far=0, dtype="bf16"),
        # one new token of each of a batch of answers
        dict(name="append_token", op="append", batch=8, new=1, ragged=False, context=2067, page=16, heads=32, kv_heads=8,
             dim=128, rot=128, interleaved=False, norm=True, cache8=False, queries=True, dtype="bf16"),
        # prompts of different lengths, small heads
        dict(name="append_prompts", op="append", batch=5, new=333, ragged=True, context=999, page=48, heads=20,
             kv_heads=4, dim=64, rot=64, interleaved=True, norm=False, cache8=False, queries=False, dtype="f16"),
        # long chunks into a cache of E4M3 codes
        dict(name="append_chunk_codes", op="append", batch=2, new=4096, ragged=False, context=8192, page=64, heads=32,
             kv_heads=8, dim=128, rot=128, interleaved=False, norm=True, cache8=True, queries=True, dtype="bf16"),
        # one new token over a short context: the smallest call
        dict(name="attn_token", op="attention", batch=1, new=1, ragged=False, context=512, lens=False, page=16, heads=32,
             kv_heads=8, dim=128, causal=True, cache8=False, codes=False, dtype="bf16"),
        # new tokens of a batch of answers over long contexts of different lengths
        dict(name="attn_tokens_long", op="attention", batch=8, new=1, ragged=False, context=20670, lens=True, page=16,
             heads=32, kv_heads=8, dim=128, causal=True, cache8=False, codes=False, dtype="bf16"),
        # the same over a cache of E4M3 codes, written as codes for the out-projection
        dict(name="attn_tokens_codes", op="attention", batch=16, new=1, ragged=False, context=20670, lens=True, page=64,
             heads=32, kv_heads=8, dim=128, causal=True, cache8=True, codes=True, dtype="bf16"),
        # a few drafted tokens of each answer, small heads, pages of 48
        dict(name="attn_drafts", op="attention", batch=7, new=5, ragged=True, context=4133, lens=True, page=48, heads=20,
             kv_heads=4, dim=64, causal=True, cache8=False, codes=False, dtype="f16"),
        # prompts of different lengths without a past
        dict(name="attn_prompts", op="attention", batch=6, new=1077, ragged=True, context=1077, lens=False, page=32,
             heads=32, kv_heads=8, dim=128, causal=True, cache8=False, codes=True, dtype="bf16"),
        # a chunk of a long prompt: the largest product
        dict(name="attn_chunk", op="attention", batch=1, new=4096, ragged=False, context=20670, lens=False, page=128,
             heads=32, kv_heads=8, dim=128, causal=True, cache8=False, codes=False, dtype="bf16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention"])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        rot = rng.choice([dim, dim, 32, 48])
        return dict(op=op, rows=_spread(rng, 1, 20670), heads=min(heads, 40), kv_heads=kv, dim=dim, rot=rot,
                    axes=rng.choice([1, 1, 3]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.6,
                    amplitude=rng.choice([1.0, 1.125]), far=rng.choice([0, 0, 1000000]), dtype=dtype)
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    if op == "append":
        dim = rng.choice([64, 80, 96, 128, 128])
        c = dict(op=op, batch=rng.choice([1, 2, 3, 5, 8, 16]), new=_spread(rng, 1, 4096), ragged=rng.random() < 0.5,
                 context=0, page=page, heads=heads, kv_heads=kv, dim=dim, rot=rng.choice([dim, dim, 32]),
                 interleaved=rng.random() < 0.4, norm=rng.random() < 0.6, cache8=rng.random() < 0.4,
                 queries=rng.random() < 0.7, dtype=dtype)
        if rng.random() < 0.3:
            c["new"] = 1
        while c["batch"] * c["new"] > 8192:
            c["new"] = (c["new"] + 1) // 2
        c["context"] = max(c["new"], _spread(rng, 1, 16384 // c["batch"]))
        return c
    c = dict(op=op, batch=rng.choice([1, 1, 2, 3, 5, 8, 16]), new=_spread(rng, 1, 4096), ragged=rng.random() < 0.4,
             context=_spread(rng, 1, 20670), lens=rng.random() < 0.5, page=page, heads=heads, kv_heads=kv,
             dim=rng.choice([64, 64, 80, 96, 128, 128]), causal=rng.random() < 0.8, cache8=rng.random() < 0.4,
             codes=rng.random() < 0.3, dtype=dtype)
    if rng.random() < 0.4:
        c["new"] = rng.choice([1, 1, 2, 5])
    while c["batch"] * c["heads"] * c["new"] * c["context"] > 32 * 4096 * 20670 // 2:
        c["new"] = (c["new"] + 1) // 2
    c["context"] = max(c["context"], c["new"])
    return c


# ------------------------------------------------------------------ inputs

def _new_lens(case):
    """New tokens of each sequence: a ragged batch has from all down to about a half."""
    n, B = case["new"], case["batch"]
    return [max(1, n - i * n // (2 * B)) if case["ragged"] else n for i in range(B)]


def _axis_pairs(case):
    """Pairs of dimensions that each axis of the positions rotates."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return (half,)
    side = half * 3 // 8
    return (half - 2 * side, side, side)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    dt = TYPES[case["dtype"]]
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]

    def normal(shape, std, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def whole(lo, hi, n):
        """n whole numbers of lo .. hi, also known on the host."""
        t = torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")
        return t.tolist()

    if case["op"] != "attention":
        half = case["rot"] // 2
        s["freqs"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        s["turns"] = None
        if own:
            import w8a16_linear_gb300 as W
            s["turns"] = W.rope_turns(s["freqs"], "cuda")
        s["freqs"] = s["freqs"].cuda()
        s["q_weight"] = (1.0 + normal((D,), 0.1)).to(dt) if case["norm"] else None
        s["k_weight"] = (1.0 + normal((D,), 0.1)).to(dt) if case["norm"] else None
    if case["op"] == "rope":
        M = case["rows"]
        # queries and keys as a shared projection writes them: one row a token
        qk = normal((M, Hq + Hk, D), 1.5, dt)
        s["q"], s["k"] = qk[:, :Hq], qk[:, Hq:]
        s["q_out"] = torch.empty((M, Hq, D), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((M, Hk, D), dtype=dt, device="cuda")
        at = torch.arange(M, device="cuda", dtype=torch.int32) + whole(0, case["far"], 1)[0]
        if case["axes"] == 3:                                # frame, row and column of each token
            at = torch.stack([at // 1590, at // 53 % 30, at % 53]).to(torch.int32).contiguous()
        s["positions"] = at
        return s

    B, page, ctx = case["batch"], case["page"], case["context"]
    new = _new_lens(case)
    if case["op"] == "append" or case["lens"]:               # between a half and all of the context
        lens = [max(n, x) for n, x in zip(new, whole((ctx + 1) // 2, ctx, B))]
    else:
        lens = [max(ctx, n) if not case["ragged"] else n + ctx - case["new"] for n in new]
    s["new_lens"], s["lens"] = new, lens
    T = sum(new)
    starts = [sum(new[:b]) for b in range(B + 1)]
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    P = (max(ctx, case["new"]) + page - 1) // page
    pages = B * P + 3
    s["page_table"] = torch.randperm(pages, generator=g, device="cuda")[:B * P].view(B, P).to(torch.int32)
    shape = (pages, page, Hk, D)
    s["k_scale"] = s["v_scale"] = None
    if case["cache8"]:
        s["k_scale"] = torch.full((1,), K_SCALE, device="cuda")
        s["v_scale"] = torch.full((1,), V_SCALE, device="cuda")
        s["k_cache"] = (normal(shape, 1.0) / K_SCALE).clamp(-448, 448).to(F8).view(torch.uint8)
        s["v_cache"] = (normal(shape, 1.0) / V_SCALE).clamp(-448, 448).to(F8).view(torch.uint8)
    else:
        s["k_cache"], s["v_cache"] = normal(shape, 1.0, dt), normal(shape, 1.0, dt)
    # of each new token: its sequence and its position there (the plain form's)
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
    pos = torch.cat([torch.arange(n) + x - n for n, x in zip(new, lens)])
    s["seq"], s["pos"] = seq.cuda(), pos.cuda()
    if case["op"] == "append":
        qkv = normal((T, Hq + 2 * Hk, D), 1.5, dt)           # as a shared projection writes them
        s["q"] = qkv[:, :Hq] if case["queries"] else None
        s["k"], s["v"] = qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        s["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda") if case["queries"] else None
        return s
    s["q"] = normal((T, Hq, D), 1.0, dt)
    s["s_out"] = torch.full((1,), OUT_SCALE, device="cuda") if case["codes"] else None
    s["out"] = torch.empty((T, Hq, D), dtype=torch.uint8 if case["codes"] else dt, device="cuda")
    n = max(new)
    at = torch.arange(n)[None, :].expand(B, n)
    s["pad"] = (torch.tensor(starts[:B])[:, None] + at).clamp(max=T - 1).cuda()   # token of each padded row
    s["rows"] = (seq * n + torch.cat([torch.arange(m) for m in new])).cuda()      # padded row of each token
    s["pad_pos"] = (torch.tensor(lens)[:, None] - torch.tensor(new)[:, None] + at).cuda()
    s["ws"] = None
    if own:
        import w8a16_linear_gb300 as W
        s["ws"] = W.paged_attention_workspace(s["q"], s["k_cache"], s["page_table"], max_q=n)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"rope": _plain_rope, "append": _plain_append, "attention": _plain_attention}[s["op"]](s)


def _run_own(s):
    import w8a16_linear_gb300 as W
    if s["op"] == "rope":
        q, k = W.qk_norm_rope(s["q"], s["k"], s["positions"], s["turns"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                              eps=EPS, interleaved=s["interleaved"], axes=_axis_pairs(s), amplitude=s["amplitude"],
                              q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    if s["op"] == "append":
        q = W.paged_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["q_start"], s["kv_len"],
                              turns=s["turns"], q=s["q"], q_weight=s["q_weight"] if s["queries"] else None,
                              k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"], k_scale=s["k_scale"],
                              v_scale=s["v_scale"], q_out=s["q_out"])
        return {"q": q, **_caches(s)}
    out = W.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["q_start"], s["kv_len"],
                            max_q=max(s["new_lens"]), causal=s["causal"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                            s_out=s["s_out"], out=s["out"], ws=s["ws"])
    return out.view(F8) if s["codes"] else out


def _caches(s):
    if s["cache8"]:
        return {"k_cache": s["k_cache"].view(F8), "v_cache": s["v_cache"].view(F8)}
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_heads(x, weight, cos, sin, rot, interleaved):
    """Norm (with a weight) and rotation of every head of x [rows, heads, D], in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight.float()
    out = x.clone() if rot < x.shape[2] else torch.empty_like(x)
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return out


def _plain_angles(positions, freqs, amplitude):
    """cos and sin [rows, 1, rot / 2]; positions [rows] or, for each pair, [rows, rot / 2]."""
    a = (positions if positions.dim() == 2 else positions[:, None]).double() * freqs
    return (a.cos() * amplitude).float()[:, None], (a.sin() * amplitude).float()[:, None]


def _pair_positions(s):
    """The position that rotates each pair: its axis's."""
    if s["axes"] == 1:
        return s["positions"]
    return torch.cat([p[:, None].expand(-1, n) for p, n in zip(s["positions"], _axis_pairs(s))], 1)


def _plain_rope(s):
    cos, sin = _plain_angles(_pair_positions(s), s["freqs"], s["amplitude"])
    dt = s["q"].dtype
    return {n: _plain_heads(s[n], s[n + "_weight"], cos, sin, s["rot"], s["interleaved"]).to(dt) for n in ("q", "k")}


def _plain_append(s):
    cos, sin = _plain_angles(s["pos"], s["freqs"], 1.0)
    page = s["page_table"][s["seq"], s["pos"] // s["page"]].long()
    slot = s["pos"] % s["page"]
    k = _plain_heads(s["k"], s["k_weight"], cos, sin, s["rot"], s["interleaved"])
    v = s["v"]
    if s["cache8"]:
        k = (k / s["k_scale"]).clamp(-448.0, 448.0).to(F8).view(torch.uint8)
        v = (v.float() / s["v_scale"]).clamp(-448.0, 448.0).to(F8).view(torch.uint8)
    s["k_cache"][page, slot] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, slot] = v
    q = None
    if s["queries"]:
        q = _plain_heads(s["q"], s["q_weight"], cos, sin, s["rot"], s["interleaved"]).to(s["q"].dtype)
    return {"q": q, **_caches(s)}


def _gathered(s, name):
    """[B, kv_heads, positions, D] of a cache, in 32 bits."""
    c = s[name + "_cache"][s["page_table"].long()]
    B, P, page, Hk, D = c.shape
    c = c.view(F8).float() * s[name + "_scale"] if s["cache8"] else c.float()
    return c.view(B, P * page, Hk, D).transpose(1, 2)


def _plain_attention(s):
    B, Hq, Hk, D = (s[k] for k in ("batch", "heads", "kv_heads", "dim"))
    G, n = Hq // Hk, s["pad"].shape[1]
    # the query heads that share a key head stand one below the other
    q = s["q"].float()[s["pad"]].view(B, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    k, v = _gathered(s, "k"), _gathered(s, "v")
    T = k.shape[2]
    p = (q @ (k * D ** -0.5).transpose(2, 3)).view(B, Hk, n, G, T)
    at = torch.arange(T, device="cuda")
    there = at[None, :] < s["kv_len"][:, None]                                   # [B, T]
    ok = there[:, None].expand(B, n, T)
    if s["causal"]:
        ok = ok & (at <= s["pad_pos"][:, :, None])
    p.masked_fill_(~ok[:, None, :, None], float("-inf"))
    p = p.sub_(p.amax(4, keepdim=True).clamp_min(-1e38)).exp_().view(B, Hk, n * G, T)
    total = p.sum(3, keepdim=True)
    o = torch.where(total > 0, (p @ v.masked_fill(~there[:, None, :, None], 0.0)) / total, 0.0)
    o = o.view(B, Hk, n, G, D).permute(0, 2, 1, 3, 4).reshape(B * n, Hq, D)[s["rows"]]
    if s["codes"]:
        return (o / s["s_out"]).clamp(-448.0, 448.0).to(F8)
    return o.to(s["q"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        M = case["rows"]
        per = 4 * (4 if case["norm"] else 0) + 3 * 4
        return {"bytes": M * (Hq + Hk) * D * 4 + 4 * M * case["axes"], "flops": M * (Hq + Hk) * D * per // 4}
    new, B = _new_lens(case), case["batch"]
    T, cell = sum(new), 1 if case["cache8"] else 2
    if case["op"] == "append":
        n = T * Hk * D * 2 * (2 + cell) + (T * Hq * D * 4 if case["queries"] else 0)
        return {"bytes": n + 4 * (2 * B + 1) + 4 * T, "flops": 7 * T * D * (Hk + (Hq if case["queries"] else 0))}
    ctx = case["context"]
    keys = pairs = 0
    for m in new:
        x = max(m, 0.75 * ctx) if case["lens"] else max(ctx, m) if not case["ragged"] else m + ctx - case["new"]
        keys += x
        pairs += m * x - (m * (m - 1) / 2 if case["causal"] else 0)
    n = T * Hq * D * (2 + (1 if case["codes"] else 2)) + 2 * keys * Hk * D * cell
    return {"bytes": n + 4 * (2 * B + 1) + 4 * keys / case["page"], "flops": 4 * Hq * D * pairs}


# ------------------------------------------------------------------ the definition, in 64 bits

def _turned(x, weight, pos, s):
    """Norm and rotation as complex numbers; pos [rows, rot / 2]."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() / (torch.linalg.vector_norm(x, dim=2, keepdim=True).square() / x.shape[2] + EPS).sqrt()
    r = s["rot"]
    pairs = x[..., :r].unflatten(2, (r // 2, 2)) if s["interleaved"] else x[..., :r].unflatten(2, (2, r // 2)).transpose(2, 3)
    angle = pos.double() * s["freqs"]
    turn = torch.polar(torch.full_like(angle, s.get("amplitude", 1.0)), angle)[:, None]
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = y.flatten(2) if s["interleaved"] else y.transpose(2, 3).flatten(2)
    return torch.cat([y, x[..., r:]], 2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        pos = _pair_positions(s)
        pos = pos if pos.dim() == 2 else pos[:, None].expand(-1, case["rot"] // 2)
        return {n: _turned(s[n], s[n + "_weight"], pos, s) for n in ("q", "k")}
    if case["op"] == "append":
        pos = s["pos"][:, None].expand(-1, case["rot"] // 2)
        k, v = _turned(s["k"], s["k_weight"], pos, s), s["v"].double()
        c = _caches(s)
        kc, vc = c["k_cache"].double(), c["v_cache"].double()
        if case["cache8"]:
            k, v = (k / K_SCALE).clamp(-448, 448), (v / V_SCALE).clamp(-448, 448)
        t = 0
        for b, (n, x) in enumerate(zip(s["new_lens"], s["lens"])):
            table = s["page_table"][b].tolist()
            at = x - n
            while at < x:                                    # the rest of a page at a time
                page, slot = table[at // case["page"]], at % case["page"]
                m = min(case["page"] - slot, x - at)
                kc[page, slot:slot + m], vc[page, slot:slot + m] = k[t:t + m], v[t:t + m]
                at, t = at + m, t + m
        q = _turned(s["q"], s["q_weight"], pos, s) if case["queries"] else None
        return {"q": q, "k_cache": kc, "v_cache": vc}
    T, Hq, D = s["q"].shape
    G = Hq // case["kv_heads"]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, x) in enumerate(zip(s["new_lens"], s["lens"])):
        at = s["page_table"][b].long()
        k, v = (s[c][at].flatten(0, 1)[:x] for c in ("k_cache", "v_cache"))
        if case["cache8"]:
            k, v = k.view(F8).double() * K_SCALE, v.view(F8).double() * V_SCALE
        later = torch.ones((n, x), dtype=torch.bool, device="cuda").triu(x - n + 1) if case["causal"] else None
        for h in range(Hq):
            e = torch.einsum("ld,td->lt", s["q"][t:t + n, h].double(), k[:, h // G].double()) / math.sqrt(D)
            if later is not None:
                e.masked_fill_(later, float("-inf"))
            out[t:t + n, h] = torch.softmax(e, dim=1) @ v[:, h // G].double()
        t += n
    return (out / OUT_SCALE).clamp(-448, 448) if case["codes"] else out
