"""What the tests of the paged cache's operators share: seeded batches and the
operators' definitions in 64 bits, on whichever device the tensors are."""

import math
from types import SimpleNamespace

import torch

F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dt):
    """Largest relative error of one rounding to dt."""
    return torch.finfo(dt).eps / 2


def smallest_half(dt):
    """Half of the smallest subnormal's step, which bounds the rounding's error below the normal range."""
    return float(torch.finfo(dt).smallest_normal) * torch.finfo(dt).eps / 2


def batch(new, lens, page, Hk, D, dtype="bf16", codes=False, seed=0, std=1.0, device="cuda", extra=3, cols=None,
          fill=None):
    """A cache whose pages are handed out in random order.  ``fill``: what the
    cells hold that belong to no position of a sequence."""
    g = torch.Generator(device=device).manual_seed(seed)
    B = len(new)
    cols = cols if cols is not None else max(1, max((n + page - 1) // page for n in lens))
    pages = B * cols + extra
    table = torch.randperm(pages, generator=g, device=device)[:B * cols].view(B, cols).to(torch.int32)
    shape = (pages, page, Hk, D)
    b = SimpleNamespace(new=list(new), lens=list(lens), page=page, B=B, T=sum(new), cols=cols, table=table, codes=codes,
                        k_scale=None, v_scale=None, dt=DT[dtype])
    k, v = (torch.randn(shape, generator=g, device=device) * std for _ in range(2))
    if codes:
        b.k_scale, b.v_scale = (torch.full((1,), s, device=device) for s in (0.03125, 0.0234375))
        b.k = (k / b.k_scale).clamp(-448, 448).to(F8).view(torch.uint8)
        b.v = (v / b.v_scale).clamp(-448, 448).to(F8).view(torch.uint8)
    else:
        b.k, b.v = k.to(b.dt), v.to(b.dt)
    if fill is not None:
        free = torch.ones((pages, page), dtype=torch.bool, device=device)
        for i, n in enumerate(lens):
            at = torch.arange(n, device=device)
            free[table[i][at // page].long(), at % page] = False
        b.k[free], b.v[free] = fill, fill
    b.q_start = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32, device=device)
    b.kv_len = torch.tensor(lens, dtype=torch.int32, device=device)
    return b


def values(b, name, i, n):
    """[n, Hk, D] in 64 bits: the cache at positions 0 .. n - 1 of sequence i (zeros where the page is none)."""
    c, s = getattr(b, name), getattr(b, name + "_scale")
    at = torch.arange(n, device=c.device)
    page = b.table[i][at // b.page].long()
    there = (page >= 0) & (page < c.shape[0])
    x = c[page.clamp(0, c.shape[0] - 1), at % b.page]
    x = x.view(F8).double() * s.double() if b.codes else x.double()
    return torch.where(there[:, None, None], x, 0.0)


def exact_attention(b, q, causal=True, scale=None, max_q=None):
    """(o, bound on the kernel's error, rows that are written); see test_gpu_paged_attention.py."""
    T, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    h = half_step(q.dtype)
    o = torch.zeros((T, H, D), dtype=torch.float64, device=q.device)
    err, written = torch.zeros_like(o), torch.zeros((T,), dtype=torch.bool, device=q.device)
    for i in range(b.B):
        t0, n, length = sum(b.new[:i]), b.new[i], b.lens[i]
        if n == 0:
            continue
        m = min(n, max_q) if max_q else n
        written[t0:t0 + m] = True
        x = max(0, min(length, b.cols * b.page))
        if x == 0:
            continue
        k, v = (values(b, c, i, x).repeat_interleave(H // b.k.shape[2], 1) for c in ("k", "v"))
        qi = q[t0:t0 + m].double()
        pos = length - n + torch.arange(m, device=q.device)
        ok = torch.arange(x, device=q.device)[None] <= (pos[:, None] if causal else x)
        last = int(pos[-1]) + 1 if causal else x
        # cells that no row sees may hold anything
        k, v = k.clone(), v.clone()
        k[max(last, 0):], v[max(last, 0):] = 0.0, 0.0
        vf = torch.where(torch.isfinite(v), v, 0.0)
        s = torch.einsum("lhd,thd->hlt", qi, k) * scale
        size = torch.einsum("lhd,thd->hlt", qi.abs(), k.abs()) * scale
        s = s.masked_fill(~ok, float("-inf"))
        some = (s > float("-inf")).any(-1, keepdim=True)
        p = torch.where(some, torch.softmax(torch.where(some, s, 0.0), -1), 0.0)
        oi = torch.einsum("hlt,thd->lhd", p, vf)
        A = torch.einsum("hlt,thd->lhd", p, vf.abs())
        size, top = size[ok.expand_as(size)], torch.where(s > float("-inf"), s.abs(), 0.0)
        size, top = (float(t.nan_to_num(0.0).max()) if t.numel() else 0.0 for t in (size, top))
        E = h + 2 * (2 * D * 2.0 ** -24 * size + 2.0 ** -22 * top * 1.45 + 2.0 ** -22) + 4 * (x + 64) * 2.0 ** -24
        e = A * E + h * (oi.abs() + A * E) + smallest_half(q.dtype)
        if h < 2.0 ** -10:
            e = e + x * 2.0 ** -25 * vf.abs().max()
        if b.codes:   # weights beside E4M3 cells: see test_gpu_paged_attention.py
            e = e + x * 2.0 ** -24 * vf.abs().max()
        # a value that is not finite and counts spoils its own column
        spoiled = torch.einsum("hlt,thd->lhd", (ok & (s > float("-inf"))).double(), (~torch.isfinite(v)).double()) > 0
        o[t0:t0 + m], err[t0:t0 + m] = torch.where(spoiled, float("nan"), oi), e
    return o, err, written


def exact_heads(x, weight, pos, freqs, eps=1e-6, interleaved=False, amplitude=1.0):
    """(y, bound on a kernel's error before the last rounding) of the norm and
    rotation of x [M, H, D] in 64 bits; pos [M, pairs]; see test_gpu_rope.py."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() / ((x * x).mean(-1, keepdim=True) + eps).sqrt()
    y, e = x.clone(), x.abs() * 2.0 ** -18
    if freqs is not None:
        r = 2 * len(freqs)
        a = pos.double() * freqs.double()
        c, s = (amplitude * a.cos())[:, None], (amplitude * a.sin())[:, None]
        first, second = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
        u, v = x[..., first], x[..., second]
        y[..., first], y[..., second] = u * c - v * s, v * c + u * s
        e[..., first] = e[..., second] = (u.abs() + v.abs()) * amplitude * 2.0 ** -17
    return y, e


def spread(v, n):
    """Positions [M] for each of n pairs."""
    return v[:, None].expand(-1, n)


def near(got, y, e):
    """Whether got (16 bits) is within e and its own rounding of y, and NaN where y is."""
    h = half_step(got.dtype)
    bad = ~((got.double() - y).abs() <= e + h * (y.abs() + e) + smallest_half(got.dtype))
    return not (bad & ~(torch.isnan(y) & torch.isnan(got))).any()


def code_near(got, y, e):
    """Whether the codes got lie between those of y - e and y + e (y in units of the codes)."""
    val = got.view(F8).cpu().double()
    lo, hi = ((y + s * e).cpu().float().clamp(-448, 448).to(F8).double() for s in (-1.0001, 1.0001))
    # the conversion to 32 bits rounds too: a step of 2^-24 is within the 1.0001 unless e is 0
    return bool((((lo <= val) & (val <= hi)) | (torch.isnan(lo) & torch.isnan(val))).all())


assert math.isclose(half_step(torch.bfloat16), 2.0 ** -8)
