"""Plain forms of a step's operators, shared by their tests: the plan as loops over whole numbers, rotary positions
and trees in 64 bits."""
from __future__ import annotations

import math

import torch


def ancestors(parents):
    """For each row of one sequence the rows above it in its tree and itself; parents: list (negative: none)."""
    rows = []
    for i, up in enumerate(parents):
        rows.append((rows[up] if 0 <= up < i else []) + [i])
    return rows


def pack(rows, words):
    """Lists of bit numbers as 32-bit words (int32)."""
    out = []
    for bits in rows:
        v = 0
        for i in bits:
            v |= 1 << i
        w = [(v >> (32 * k)) & 0xffffffff for k in range(words)]
        out.append([x - (1 << 32) if x >> 31 else x for x in w])
    return torch.tensor(out, dtype=torch.int32).reshape(len(rows), words)


def random_tree(n, g, chain=0.3):
    u = torch.rand(3, max(n, 1), generator=g).tolist()
    return [-1 if i == 0 or u[0][i] < 0.1 else (i - 1 if u[1][i] < chain else int(u[2][i] * i)) for i in range(n)]


def plan(new_lens, total, old, table, free, count, page, parents=None, words=0):
    """What cache_plan leaves: dict of lists and tensors.  table: list of lists (copied)."""
    table = [list(r) for r in table]
    cap = len(table[0])
    cu = [0]
    for n in new_lens:
        cu.append(min(cu[-1] + max(n, 0), total))
    out = {"cu": cu, "slots": [-1] * total, "positions": [0] * total, "unplaced": [], "seqlens": [], "table": table,
           "masks": torch.zeros(total, max(words, 1), dtype=torch.int32)}
    upto, taken = 0, 0
    for b in range(len(new_lens)):
        n, at = cu[b + 1] - cu[b], min(max(old[b], 0), cap * page)
        have, want = -(-at // page), -(-(at + n) // page)
        need = want - have if want <= cap else 0
        upto += need
        given = want <= cap and (need == 0 or upto <= count)
        new = {}
        for k in range(have, want):
            new[k] = free[count - 1 - (upto - need) - (k - have)] if given else -1
            if k < cap:
                table[b][k] = new[k]
        if given and need:
            taken = upto
        lost = 0
        rows = ancestors((parents[cu[b]:cu[b + 1]] if parents is not None else [])[:32 * words])
        for i in range(n):
            pos, k = at + i, (at + i) // page
            of = table[b][k] if k < have else new[k]
            if k >= cap:
                of = -1
            out["slots"][cu[b] + i] = -1 if of < 0 else of * page + pos % page
            lost += of < 0
            depth = i
            if parents is not None:
                depth = len(rows[i]) - 1 if i < len(rows) else 0
            out["positions"][cu[b] + i] = at + depth
        if parents is not None:
            out["masks"][cu[b]:cu[b] + len(rows)] = pack(rows, words)
        out["unplaced"].append(lost)
        out["seqlens"].append(at + n)
    out["count"] = count - taken
    return out


def turned(x, angle, rot, interleaved, scale, back=False):
    """(y, size) in 64 bits: rows x [rows, heads, dim] turned by angle [rows, rot / 2]; size bounds what a relative
    error of the sines, cosines and products counts for."""
    x = x.double()
    cos, sin = (scale * torch.cos(angle))[:, None], ((-scale if back else scale) * torch.sin(angle))[:, None]
    y, size = x.clone(), torch.zeros_like(x)
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        ya, yb = y[..., 0:rot:2], y[..., 1:rot:2]
        sa, sb = size[..., 0:rot:2], size[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        ya, yb = y[..., :rot // 2], y[..., rot // 2:rot]
        sa, sb = size[..., :rot // 2], size[..., rot // 2:rot]
    ya.copy_(a * cos - b * sin)
    yb.copy_(b * cos + a * sin)
    sa.copy_(abs(scale) * (a.abs() + b.abs()))
    sb.copy_(sa)
    return y, size


def angles(positions, turns):
    """position * turns / 2^64 of a turn, reduced in whole numbers, in radians (float64)."""
    return torch.tensor([[2 * math.pi * (((p * t) % (1 << 64)) / 2 ** 64) for t in turns] for p in positions],
                        dtype=torch.float64)


def attend_tree(q, k, v, scale, seen):
    """attend of paged_cases for a mask seen [n, keys]."""
    n, H, D = q.shape
    group = H // k.shape[1]
    q = q.double()
    out = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device=q.device)
    A, S = torch.zeros_like(out), torch.zeros_like(lse)
    if n == 0 or k.shape[0] == 0:
        return out, lse, A, S
    some = seen.any(0)  # keys that nobody sees may hold anything
    k, v = (torch.where(some[:, None, None], x, torch.zeros_like(x)) for x in (k, v))
    for h in range(H):
        kk, vv = k[:, h // group], v[:, h // group]
        x = torch.where(seen, scale * (q[:, h] @ kk.T), torch.full((), -math.inf, dtype=torch.float64, device=q.device))
        y = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(y > -math.inf, y, torch.zeros_like(y))[:, None])
        out[:, h], lse[h], A[:, h] = p @ vv, y, p @ vv.abs()
        S[h] = torch.where(seen, scale * (q[:, h].abs() @ kk.abs().T), torch.zeros_like(x)).amax(-1)
    return out, lse, A, S
