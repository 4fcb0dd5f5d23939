"""Inputs, layouts and the plain 64-bit forms shared by the paged-cache tests."""
from __future__ import annotations

import math

import torch

E4M3_MAX = 448.0


def cu_of(lens, device):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=device)


def quantise(x):
    """(codes [..., D] float8_e4m3fn, scale [...] bf16) of bf16 x: the least power of two s >= 2^-127 with
    amax <= 448 s, computed in 64 bits."""
    x = x.double()
    amax = x.abs().amax(-1)
    s = torch.exp2(torch.clamp(torch.ceil(torch.log2(amax / E4M3_MAX)), min=-127.0))
    s = torch.where(amax > 0, s, torch.ones_like(s))
    bad = ~torch.isfinite(amax)
    s = torch.where(bad, torch.full_like(s, math.nan), s)
    y = torch.where(bad[..., None], torch.zeros_like(x), x / torch.where(bad, torch.ones_like(s), s)[..., None])
    return torch.clamp(y, -E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn), s.to(torch.bfloat16)


def make_cache(lens, heads, dim, page, kind, device, seed=0, order="nhd", spare=3, amp=1.0, fill=None, columns=1):
    """A PagedCache of random pages in random order with lens[b] positions each; pages no sequence uses and rows
    past a sequence's end hold NaN (bf16) or NaN scales.  Returns (cache, k, v): lists of [lens[b], heads, dim]
    float64 held values."""
    from packed_variable_length_varlen_gb300 import varlen_attn as va
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    width = max(need + [columns])
    perm = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n

    def pool(dtype, value):
        if order == "hnd":
            return torch.full((pages, heads, page, dim), value, device=device).to(dtype).transpose(1, 2)
        if order == "padded":
            return torch.full((pages, page, heads * 2, dim + 32), value, device=device).to(dtype)[:, :, ::2, :dim]
        return torch.full((pages, page, heads, dim), value, device=device).to(dtype)

    if order == "together":  # K and V of a page side by side
        both = torch.full((pages, 2, page, heads, dim), math.nan if kind == "bf16" else 1.0, device=device)
        both = both.to(torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
        pools = [both[:, 0], both[:, 1]]
    else:
        pools = [pool(torch.bfloat16, math.nan) if kind == "bf16" else pool(torch.float8_e4m3fn, 1.0) for _ in range(2)]
    scales = [None if kind == "bf16" else torch.full((pages, heads, page), math.nan, dtype=torch.bfloat16,
                                                     device=device) for _ in range(2)]
    held = [[], []]
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        pg, row = table[b].long()[pos // page].to(device), (pos % page).to(device)
        for i in range(2):
            x = (torch.randn(n, heads, dim, generator=g) * amp).to(torch.bfloat16).to(device)
            if fill is not None:
                x = fill(x, b, i)
            if kind == "bf16":
                pools[i][pg, row] = x
                held[i].append(x.double())
            else:
                codes, s = quantise(x)
                pools[i].view(torch.uint8)[pg, row] = codes.view(torch.uint8)
                scales[i][pg, :, row] = s
                held[i].append(codes.double() * s.double()[..., None])
    cache = va.PagedCache(pools[0], pools[1], table.to(device), torch.tensor(lens, dtype=torch.int32, device=device),
                          scales[0], scales[1])
    return cache, held[0], held[1]


def attend(q, k, v, scale, left, right):
    """(O, LSE, A, S) of one segment in 64 bits: q [n, H, D], k / v [m, Hk, D]; A = sum_j p_j |v_j| per element,
    S = the largest scale * sum_d |q_d k_d| of a row's visible keys (0 when none)."""
    n, H, D = q.shape
    m = k.shape[0]
    group = H // k.shape[1]
    q = q.double()
    out = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device=q.device)
    A, S = torch.zeros_like(out), torch.zeros_like(lse)
    if n == 0 or m == 0:
        return out, lse, A, S
    i = torch.arange(n, device=q.device)[:, None] + (m - n)
    j = torch.arange(m, device=q.device)[None]
    seen = torch.ones(n, m, dtype=torch.bool, device=q.device)
    if left >= 0:
        seen &= j >= i - left
    if right >= 0:
        seen &= j <= i + right
    for h in range(H):
        kk, vv = k[:, h // group], v[:, h // group]
        x = scale * (q[:, h] @ kk.T)
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        y = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(y > -math.inf, y, torch.zeros_like(y))[:, None])
        out[:, h], lse[h], A[:, h] = p @ vv, y, p @ vv.abs()
        S[h] = torch.where(seen, scale * (q[:, h].abs() @ kk.abs().T), torch.zeros_like(x)).amax(-1)
    return out, lse, A, S


def check_attend(out, lse, ref, dim, keys):
    """Bounds from the roundings: P to bf16 (2^-8 relative per weight, so 2^-8 A), O to bf16 (2^-8 |O| and A covers
    the P error's own share); the score's fp32 sum of D products (D 2^-24 relative to the sum of |q k|, S) and
    its product with scale * log2 e, and exp2's 2^-22, which move a weight by a relative e and its row sum by the
    same; sums of `keys` fp32 terms in parts of at least 16 (keys / 16 + 64) 2^-24."""
    o, l, A, S = ref
    e = (dim + 8) * 2.0 ** -24 * S.T[..., None] + 2.0 ** -21 + (keys / 16 + 64) * 2.0 ** -24
    tol = 2.0 ** -8 * (A + o.abs()) + (2 * e + 2.0 ** -15) * A + 1e-30
    d = (out.double() - o).abs()
    assert torch.isfinite(out).all()
    assert (d <= tol).all(), "O off by %.3g where %.3g is allowed (worst ratio %.3g)" % (
        d.max(), tol[d == d.max()].max(), (d / tol).max())
    fin = l > -math.inf
    assert torch.equal(lse[~fin].double(), l[~fin])
    el = (dim + 8) * 2.0 ** -24 * S + (keys / 16 + 64) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * torch.where(fin, l.abs(), torch.zeros_like(l))
    dl = (lse.double() - l).abs()[fin]
    assert (dl <= el[fin]).all(), "LSE off by %.3g (worst ratio %.3g)" % (dl.max(), (dl / el[fin]).max())
