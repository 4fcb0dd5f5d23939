"""Cases of what stands around the paged attention in one step of a program that generates, and in training.

Five operators, as a step that verifies drafted trees uses them one after another:

* ``plan``   -- from each request's number of new rows, built on the GPU: cu_seqlens, pages taken from the free list
  into the block table, lengths, the slot and the position of every new row, and for trees the rows' masks;
* ``write``  -- queries and keys are turned to their positions, the keys and the values go to their slots of the cache;
* ``tree``   -- attention over the pages for rows that see all of the context and those new rows that their mask names;
* ``accept`` -- the rows of the accepted path move behind the context, lengths shrink, pages go back to the free list;
* ``rotate`` -- rotary positions on packed rows, forward and gradient, for prompts and training.

``own`` chooses between a plain form in elementary torch operations and the library's entry points.  A case gives the
ranges of its lengths and a number ``shape`` that they are drawn from; values, trees and page order come from the seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _case(name, op, shape, seqs, new, ctx, heads=1, kv_heads=1, dim=64, page=16, kind="bf16", rot=0, inter=False, base=10000.0,
          stretch=1.0, far=0, grad=False, pad=0, left=-1, trees=False, caches=1, short=0):
    return {"name": name, "op": op, "type": kind, "shape": shape, "seqs": seqs, "new_lo": new[0], "new_hi": new[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "rot": rot,
            "inter": inter, "base": base, "stretch": stretch, "far": far, "grad": grad, "pad": pad, "left": left, "trees": trees,
            "caches": caches, "short": short}


def listed():
    return [
        # queries and keys of the ragged workload's prompts (64 of up to 8192 rows) before packed attention
        _case("rotate_prompts", "rotate", 1, 64, (0, 8192), (0, 0), 32, 8, 128, rot=128),
        # training, the strided workload's form: gradients of neighbouring pairs in half of each head, gaps between rows, far positions, angles stretched eightfold
        _case("rotate_grads", "rotate", 2, 2, (9001, 20011), (0, 0), 16, 16, 96, rot=48, inter=True, base=500000.0, stretch=8.0,
              far=185619, grad=True, pad=32),
        # the new rows of one decoding step of a small batch: latency
        _case("write_tokens_e4m3", "write", 3, 16, (1, 1), (1, 2000), 32, 8, 128, 16, "e4m3", rot=128),
        # chunks of four prompts over what came before
        _case("write_chunks_bf16", "write", 4, 4, (1500, 2048), (4096, 16384), 32, 8, 128, 64, rot=128, base=1000000.0),
        # one decoding step of a full batch: a token each, some at the end of a page
        _case("plan_tokens", "plan", 5, 64, (1, 1), (1, 8192), page=16),
        # the ragged workload's prompts into an empty cache
        _case("plan_prompts", "plan", 6, 64, (0, 8192), (0, 0), page=64),
        # a drafted tree for each sequence of a full batch
        _case("plan_trees", "plan", 7, 64, (16, 64), (1, 8192), page=16, trees=True),
        # four small trees under a sliding window: latency
        _case("tree_window_bf16", "tree", 8, 4, (13, 13), (500, 4000), 16, 4, 64, 16, left=1023),
        # a tree for each sequence of a full batch at ragged lengths
        _case("tree_batch_e4m3", "tree", 9, 64, (16, 64), (1, 8192), 32, 8, 128, 64, "e4m3"),
        # one large tree at the end of the long workload, seven query heads to a key head
        _case("tree_long_bf16", "tree", 10, 1, (256, 256), (77000, 77000), 56, 8, 128, 128),
        # the accepted paths of a batch in one layer's cache: latency
        _case("accept_e4m3", "accept", 11, 64, (16, 64), (1, 2000), 32, 8, 128, 16, "e4m3"),
        # the same for a large batch and four layers, as many key heads as query heads
        _case("accept_layers_bf16", "accept", 12, 256, (16, 64), (1, 300), 56, 56, 128, 16, caches=4),
    ]


def _lens(case):
    """[(new rows, rows in the cache before them)] of every sequence."""
    r = random.Random(1000 + case["shape"])
    got = [(r.randint(case["new_lo"], case["new_hi"]), r.randint(case["ctx_lo"], case["ctx_hi"])) for _ in range(case["seqs"])]
    return got


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("rotate", "write", "plan", "tree", "tree", "accept"))
    while True:
        seqs, shape = _spread(rng, 1, 256), rng.randrange(1 << 20)
        kv, group = rng.choice((1, 2, 3, 4, 8, 16, 32, 56)), rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
        kind, page, dim = rng.choice(("bf16", "e4m3")), rng.choice((16, 32, 64, 128, 256)), rng.choice((64, 96, 128))
        trees = op in ("tree", "accept") or (op == "plan" and rng.random() < 0.5)
        new_hi = _spread(rng, 1, 300 if trees else 20011)
        new = (rng.randint(0 if op == "rotate" else 1, new_hi), new_hi)
        hi = _spread(rng, 16, 77000 if op == "tree" else 8192)
        rot = 8 * rng.randint(1, dim // 8)
        case = _case("", op, shape, seqs, new, (rng.randint(0, hi), hi), kv * group, kv, dim, page, kind,
                     rot=rot if op in ("rotate", "write") else 0, inter=rng.random() < 0.5, base=rng.choice((10000.0, 500000.0, 1000000.0)),
                     stretch=rng.choice((1.0, 4.0, 8.0)), far=rng.choice((0, 0, _spread(rng, 1, 1 << 24))), grad=rng.random() < 0.5,
                     pad=rng.choice((0, 0, 8, 32)), left=rng.choice((-1, -1, _spread(rng, 32, 8192))) if op == "tree" else -1,
                     trees=trees and op == "plan", caches=rng.randint(1, 4) if op == "accept" else 1,
                     short=rng.randint(0, 64) if op == "plan" and rng.random() < 0.3 else 0)
        del case["name"]
        w, rows = work(case), sum(n for n, _ in _lens(case))
        held = sum(-(-(n + c) // page) * page for n, c in _lens(case)) * kv * dim * 4 * case["caches"]
        if rows == 0 or kv * group > 64 or w["bytes"] > 4e9 or w["flops"] > 5.5e11 or (op not in ("plan", "rotate") and held > 5.8e9):
            continue
        if op == "tree" and seqs * kv * group * max(n for n, _ in _lens(case)) * max(n + c for n, c in _lens(case)) > 1.1e9:
            continue
        if op == "write" and kind == "e4m3" and rows * kv > 60000:
            continue
        return case


def _row_bytes(case):
    """Bytes of one row of one key head in the cache: K or V."""
    return case["dim"] * 2 if case["type"] == "bf16" else case["dim"] + 2


def _words(case):
    """32-bit words of a row's mask."""
    return -(-max(n for n, _ in _lens(case)) // 32)


def work(case):
    lens, kv, dim, op = _lens(case), case["kv_heads"], case["dim"], case["op"]
    rows, turned = sum(n for n, _ in lens), case["heads"] + case["kv_heads"]
    if op == "rotate":
        return {"bytes": rows * (4 * dim * turned + 4), "flops": 3 * rows * turned * case["rot"]}
    if op == "write":
        return {"bytes": rows * (4 * dim * case["heads"] + kv * (4 * dim + 2 * _row_bytes(case)) + 12), "flops": 3 * rows * turned * case["rot"]}
    if op == "plan":
        taken = sum(-(-(n + c) // case["page"]) - -(-c // case["page"]) for n, c in lens)
        return {"bytes": len(lens) * 24 + 8 * taken + rows * (12 + (4 + 4 * _words(case) if case["trees"] else 0)), "flops": 0}
    if op == "accept":  # a path of a random tree is about as long as twice the logarithm of its size
        moved = sum(min(n, 1 + int(2 * math.log(n + 1))) for n, _ in lens)
        return {"bytes": case["caches"] * moved * kv * 4 * _row_bytes(case) + 4 * moved + len(lens) * 16, "flops": 0}
    keys = sum((min(c, case["left"]) if case["left"] >= 0 else c) + n for n, c in lens)
    pairs = sum(n * ((min(c, case["left"]) if case["left"] >= 0 else c) + 1) for n, c in lens)
    return {"bytes": 2 * keys * kv * _row_bytes(case) + rows * (case["heads"] * (4 * dim + 4) + 4 * _words(case)), "flops": 4 * pairs * case["heads"] * dim}


# ------------------------------------------------------------------ inputs

def _hold(x):
    """(codes as their values, scale) of rows x [..., dim]: scale the least power of two with amax <= 448 * scale (1 for
    rows of zeros), code = x / scale rounded to E4M3."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.clamp(e - 9 + (m > 0.875), min=-127)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    return torch.clamp(x / scale[..., None], -E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn), scale.to(torch.bfloat16)


def _ancestors(parents, inside):
    """[seqs, n, n]: whether column j is row i or above it in its tree; parents [seqs, n] (negative: none)."""
    n = parents.shape[1]
    at = torch.arange(n, device="cuda")
    step = (parents[..., None] == at) & inside[..., None]
    a = ((at[:, None] == at) & inside[..., None]) | step
    a, reach = a.float(), 1
    while reach < n:  # twice as far each time
        a, reach = ((a @ a) > 0).float(), 2 * reach
    return a > 0


def _pack(a, words):
    """Truth values [..., n] as 32-bit words [..., words]."""
    a = torch.nn.functional.pad(a, (0, 32 * words - a.shape[-1])).unflatten(-1, (words, 32)).long()
    v = (a << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    lens, heads, kv, dim, page, op = _lens(case), case["heads"], case["kv_heads"], case["dim"], case["page"], case["op"]
    total, max_new = sum(n for n, _ in lens), max(n for n, _ in lens)
    s = {"case": case, "total": total, "max_new": max_new, "max_keys": max(n + c for n, c in lens), "words": _words(case)}

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def rows(h):  # packed rows, with a gap behind each where the case has one
        x = torch.randn(total, h * dim + case["pad"], generator=g, device="cuda").to(torch.bfloat16)
        return x[:, :h * dim].unflatten(1, (h, dim))

    s["new_lens"] = ints([n for n, _ in lens])
    s["cu"] = ints([0] + [n for n, _ in lens]).cumsum(0, dtype=torch.int32)
    if case["rot"]:
        # slow pairs are stretched, fast ones are kept, as for contexts longer than the ones trained on
        f = case["base"] ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        keep = torch.clamp((f * 8192 / (2 * math.pi) - 1) / 31, 0, 1)
        s["freq"] = f * keep + f / case["stretch"] * (1 - keep)
        s["amp"] = 1.0 if case["stretch"] == 1 else 0.1 * math.log(case["stretch"]) + 1
    local = torch.arange(total, device="cuda") - s["cu"][:-1].long().repeat_interleave(s["new_lens"].long(), output_size=total)
    if op == "rotate":
        s["q"], s["k"] = rows(heads), rows(kv)
        s["positions"] = (local + torch.randint(0, case["far"] + 1, (1,), generator=g, device="cuda")).to(torch.int32) if case["far"] else None
        return s
    # trees: each row continues the one before it or a random one, now and then nothing but the context
    u = torch.rand(2, total, generator=g, device="cuda")
    parents = torch.where(u[0] < 0.3, local - 1, torch.where(u[0] < 0.95, (u[1] * local).long(), torch.full_like(local, -1)))
    s["parents"] = torch.where(local == 0, torch.full_like(local, -1), parents).to(torch.int32)
    ctx = ints([c for _, c in lens])
    have = [-(-c // page) for _, c in lens]
    want = [-(-(n + c) // page) for n, c in lens]
    pages = sum(want) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    owned = sum(have) if op == "plan" else sum(want)
    use = torch.tensor(have if op == "plan" else want, device="cuda")
    col = torch.arange(max(want), device="cuda")
    first = (use.cumsum(0) - use)[:, None]
    s["table"] = torch.where(col < use[:, None], order[(first + col).clamp(max=pages - 1)], torch.zeros_like(order[:1]))
    s["pages"] = pages
    s["free"] = torch.cat([order[owned:], torch.zeros_like(order[:owned])])  # a stack of pages nobody has
    s["free_count"] = ints([max(0, pages - owned - case["short"])])
    s["free_count_out"] = torch.zeros_like(s["free_count"])
    s["seqlens"] = ctx if op == "plan" else ctx + s["new_lens"]
    s["seqlens_out"] = torch.zeros_like(ctx)
    if op == "plan":
        s["room"] = -(-total // 64) * 64  # rows of the step's buffers
        s["parents"] = torch.nn.functional.pad(s["parents"], (0, s["room"] - total), value=-1) if case["trees"] else None
        return s
    inside = torch.arange(max_new, device="cuda") < s["new_lens"][:, None]
    row_of = (s["cu"][:-1].long()[:, None] + torch.arange(max_new, device="cuda")).clamp(max=total - 1)
    start = ctx.long().repeat_interleave(s["new_lens"].long(), output_size=total)
    if op in ("tree", "accept"):
        above = _ancestors(s["parents"].long()[row_of], inside)
        s["positions"] = (start + above.sum(-1)[inside] - 1).to(torch.int32)
        if op == "tree":
            s["masks"] = _pack(above[inside], s["words"])
        else:  # the path to a random row
            leaf = (torch.rand(len(lens), generator=g, device="cuda") * s["new_lens"]).long()
            path = above.gather(1, leaf[:, None, None].expand(-1, 1, max_new))[:, 0]
            s["kept_lens"] = path.sum(-1).to(torch.int32)
            most = int(s["kept_lens"].max())
            s["kept"] = torch.argsort((~path).to(torch.uint8), dim=1, stable=True)[:, :most].to(torch.int32).contiguous()
    else:
        s["positions"] = (start + local).to(torch.int32)
    at = s["seqlens"].long().repeat_interleave(s["new_lens"].long(), output_size=total) - s["new_lens"].long().repeat_interleave(
        s["new_lens"].long(), output_size=total) + local
    b = torch.arange(len(lens), device="cuda").repeat_interleave(s["new_lens"].long(), output_size=total)
    s["slots"] = s["table"][b, at // page].long() * page + at % page
    s["layers"] = []
    for _ in range(case["caches"]):
        layer = {}
        for name in ("k", "v"):
            x = torch.zeros(pages, page, kv, dim, device="cuda") if op == "write" else torch.randn(pages, page, kv, dim, generator=g, device="cuda")
            if case["type"] == "bf16":
                layer[name], layer[name + "_scale"] = x.to(torch.bfloat16), None
            else:  # heads and tokens differ in size, as keys and values do
                size = torch.exp2(torch.randint(-3, 3, x.shape[:3], generator=g, device="cuda").float())
                codes, scale = _hold((x * size[..., None]).to(torch.bfloat16).float())
                layer[name], layer[name + "_scale"] = codes, scale.transpose(1, 2).contiguous()
            del x
        s["layers"].append(layer)
    if op == "write":
        s["q"], s["k"], s["v"] = rows(heads), rows(kv), rows(kv)
    if op == "tree":
        s["q"] = torch.randn(total, heads, dim, generator=g, device="cuda").to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ the plain form

def _segments(cu, total):
    """(segment, row in it) of every packed row."""
    row = torch.arange(total, device="cuda")
    b = torch.searchsorted(cu[1:].long(), row, right=True)
    return b, row - cu[b.clamp(max=cu.numel() - 2)]


def _turn(x, positions, s, back=False):
    """Rows x [rows, heads, dim] turned to their positions, rounded once.  Angles are in 64 bits (positions are far), and
    so are the products before a scale for 8 bits is chosen (the largest value may lie next to where it changes)."""
    case = s["case"]
    bits = torch.float64 if case["op"] == "write" and case["type"] == "e4m3" else torch.float32
    angle = positions.double()[:, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["amp"])[:, None].to(bits), (torch.sin(angle) * (-s["amp"] if back else s["amp"]))[:, None].to(bits)
    r, rest = x[..., :case["rot"]].to(bits), x[..., case["rot"]:]
    if case["inter"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r.chunk(2, -1)
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r.to(x.dtype), rest], -1)


def _write(s):
    layer, page = s["layers"][0], s["case"]["page"]
    q, k = _turn(s["q"], s["positions"], s), _turn(s["k"], s["positions"], s)
    of, row = s["slots"] // page, s["slots"] % page
    for name, x in (("k", k), ("v", s["v"])):
        if layer[name + "_scale"] is None:
            layer[name][of, row] = x
        else:
            codes, scale = _hold(x.float())
            layer[name].view(torch.uint8)[of, row] = codes.view(torch.uint8)
            layer[name + "_scale"][of, :, row] = scale
    return {"q": q, **layer}


def _plan(s):
    page, room, table, free = s["case"]["page"], s["room"], s["table"], s["free"]
    cap, width, count = s["pages"], table.shape[1], s["free_count"].long()
    old = s["seqlens"].long().clamp(0, width * page)
    cu = torch.cat([torch.zeros_like(old[:1]), s["new_lens"].long().clamp(min=0).cumsum(0)]).clamp(max=room)
    n = cu[1:] - cu[:-1]
    have, want = (old + page - 1) // page, (old + n + page - 1) // page
    need = torch.where(want <= width, want - have, torch.zeros_like(have))
    upto = need.cumsum(0)
    given = (want <= width) & ((need == 0) | (upto <= count))
    first = upto - need
    s["free_count_out"].copy_(count - torch.where(given, upto, torch.zeros_like(upto)).clamp(max=count).amax())
    col = torch.arange(width, device="cuda")
    page_of = free[(count - 1 - first[:, None] - (col - have[:, None])).clamp(0, cap - 1)]
    new = (col >= have[:, None]) & (col < want[:, None])
    table.copy_(torch.where(new, torch.where(given[:, None], page_of, torch.full_like(page_of, -1)), table))
    s["seqlens_out"].copy_(old + n)
    b, i = _segments(cu, room)
    inside = b < n.numel()
    b = b.clamp(max=n.numel() - 1)
    at = old[b] + i
    of = table[b, (at // page).clamp(max=width - 1)].long()
    ok = inside & (given[b] | (at // page < have[b]))
    slots = torch.where(ok, of * page + at % page, torch.full_like(of, -1))
    unplaced = torch.where(given, torch.zeros_like(n), (old + n - torch.maximum(old, have * page)).clamp(min=0))
    out = {"cu": cu.to(torch.int32), "seqlens": s["seqlens_out"], "table": table, "free_count": s["free_count_out"], "slots": slots,
           "unplaced": unplaced.to(torch.int32)}
    if s["parents"] is None:
        return {**out, "positions": torch.where(inside, at, torch.zeros_like(at)).to(torch.int32)}
    t = torch.arange(s["max_new"], device="cuda")
    there = t < n[:, None]
    above = _ancestors(s["parents"].long()[(cu[:-1, None] + t).clamp(max=room - 1)], there)
    masks = torch.zeros(room, s["words"], dtype=torch.int32, device="cuda")
    masks[inside] = _pack(above[there], s["words"])
    depth = torch.zeros(room, dtype=torch.long, device="cuda")
    depth[inside] = above.sum(-1)[there] - 1
    return {**out, "positions": torch.where(inside, old[b] + depth, torch.zeros_like(at)).to(torch.int32), "masks": masks}


def _accept(s):
    page, n = s["case"]["page"], s["new_lens"].long()
    start = s["seqlens"].long() - n
    i = torch.arange(s["kept"].shape[1], device="cuda")
    there = i < s["kept_lens"][:, None]
    b = torch.arange(n.numel(), device="cuda")[:, None].expand(-1, i.numel())[there]
    src, dst = (start[:, None] + s["kept"])[there], (start[:, None] + i)[there]
    sp, dp = s["table"][b, src // page].long(), s["table"][b, dst // page].long()
    for layer in s["layers"]:
        for name in ("k", "v"):
            x = layer[name].view(torch.uint8) if layer[name + "_scale"] is not None else layer[name]
            x[dp, dst % page] = x[sp, src % page]
            if layer[name + "_scale"] is not None:
                x = layer[name + "_scale"]
                x[dp, :, dst % page] = x[sp, :, src % page]
    # pages past the new length go back, the last sequence's last page first
    left = start + s["kept_lens"]
    have, keep = (s["seqlens"].long() + page - 1) // page, (left + page - 1) // page
    col = torch.arange(s["table"].shape[1], device="cuda")
    back = s["table"].flip(0, 1)[((col >= keep[:, None]) & (col < have[:, None])).flip(0, 1)]
    at = s["free_count"].long() + torch.arange(back.numel(), device="cuda")
    s["free"][at] = back
    s["seqlens_out"].copy_(left)
    s["free_count_out"].copy_(s["free_count"] + back.numel())
    return _accepted(s)


def _accepted(s):
    return {"layers": s["layers"], "seqlens": s["seqlens_out"], "free": s["free"], "free_count": s["free_count_out"]}


def _values(s, name, page, row):
    """Cache rows [..., kv heads, dim] in 32 bits."""
    pages, scales = s["layers"][0][name], s["layers"][0][name + "_scale"]
    if scales is None:
        return pages[page, row].float()
    return pages.view(torch.uint8)[page, row].view(torch.float8_e4m3fn).float() * scales.transpose(1, 2)[page, row].float()[..., None]


def _attend(s):
    case, group = s["case"], s["case"]["heads"] // s["case"]["kv_heads"]
    t, j = torch.arange(s["max_new"], device="cuda"), torch.arange(s["max_keys"], device="cuda")
    new, keys = s["new_lens"].long(), s["seqlens"].long()
    inside = t < new[:, None]
    packed = (s["cu"][:-1].long()[:, None] + t)[inside]

    def padded(x, fill):  # packed rows as [seqs, rows, ...]
        y = torch.full((case["seqs"], s["max_new"]) + x.shape[1:], fill, dtype=x.dtype, device="cuda")
        y[inside] = x[packed]
        return y

    # queries [seqs, kv heads, rows * group, dim]
    q = padded(s["q"].float(), 0.0).unflatten(2, (case["kv_heads"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    page, row = s["table"][:, j // case["page"]].long(), (j % case["page"]).expand(case["seqs"], -1)
    x = (q @ _values(s, "k", page, row).permute(0, 2, 3, 1)) * (1.0 / math.sqrt(case["dim"]))
    # context as far back as the window reaches from the row's position, and of the new rows those in the mask
    rel = j[None] - (keys - new)[:, None]
    bits = padded(s["masks"].long(), 0).gather(2, (rel.clamp(0, 32 * s["words"] - 1) // 32)[:, None].expand(-1, s["max_new"], -1))
    seen = (((bits >> (rel.clamp(min=0) % 32)[:, None]) & 1) > 0) & (rel >= 0)[:, None] & (rel < new[:, None])[:, None]
    context = (rel < 0)[:, None].expand_as(seen)
    if case["left"] >= 0:
        context = context & (j >= padded(s["positions"].long(), 0)[..., None] - case["left"])
    x.masked_fill_(~(seen | context).repeat_interleave(group, 1)[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x @ _values(s, "v", page, row).transpose(1, 2)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + total.log()

    def back(y):  # [seqs, kv heads, rows * group, n] -> [packed rows, heads, n]
        return y.unflatten(2, (s["max_new"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)[inside]

    return {"out": back(out).to(torch.bfloat16), "lse": back(lse)[..., 0].T.contiguous()}


def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "rotate":
        at = s["positions"] if s["positions"] is not None else _segments(s["cu"], s["total"])[1]
        return {"q": _turn(s["q"], at, s, case["grad"]), "k": _turn(s["k"], at, s, case["grad"])}
    return {"write": _write, "plan": _plan, "tree": _attend, "accept": _accept}[op](s)


def _run_own(s, op):
    from packed_variable_length_varlen_gb300 import varlen_attn as va
    case = s["case"]
    if "kept_handles" not in s:  # what a program keeps beside its tensors
        s["kept_handles"] = True
        if case["rot"]:
            s["rope"] = va.Rotary(s["freq"], interleaved=case["inter"], scale=s["amp"])
        if op in ("plan", "accept"):
            s["pool"] = va.PagePool(s["table"], s["seqlens"], s["free"], s["free_count"], case["page"], s["seqlens_out"], s["free_count_out"])
        if op == "plan":
            s["plan"] = va.StepPlan(case["seqs"], s["room"], "cuda", mask_words=s["words"] if case["trees"] else 0)
        if op in ("write", "tree", "accept"):
            s["held"] = [va.PagedCache(c["k"], c["v"], s["table"], s["seqlens"], c["k_scale"], c["v_scale"]) for c in s["layers"]]
    if op == "rotate":
        turn = va.rotary_bwd if case["grad"] else va.rotary
        q, k = turn(s["q"], s["k"], s["rope"], positions=s["positions"], cu_seqlens=s["cu"] if s["positions"] is None else None)
        return {"q": q, "k": k}
    if op == "write":
        q = va.rotary_cache_write(s["held"][0], s["q"], s["k"], s["v"], s["rope"], s["positions"], s["slots"])
        return {"q": q, **s["layers"][0]}
    if op == "plan":
        p = va.cache_plan(s["pool"], s["plan"], s["new_lens"], parents=s["parents"])
        out = {"cu": p.cu_seqlens, "seqlens": s["seqlens_out"], "table": s["table"], "free_count": s["free_count_out"], "slots": p.slots,
               "unplaced": p.unplaced, "positions": p.positions}
        return {**out, "masks": p.masks} if case["trees"] else out
    if op == "accept":
        va.cache_move(s["held"], s["cu"], s["kept"], s["kept_lens"])
        va.cache_trim(s["pool"], s["kept_lens"], s["cu"])
        return _accepted(s)
    out, lse = va.attention_fwd_paged_tree(s["q"], s["held"][0], s["cu"], s["masks"], max_seqlen_q=s["max_new"], window_left=case["left"],
                                           positions=s["positions"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("plan", "accept"):  # whole numbers, and rows as they were
        return None
    s = prepare(case, seed)
    lens, page, cu = _lens(case), case["page"], s["cu"].tolist()

    def turned(x, at, sign):
        """As products with unit complex numbers."""
        x = x.double()
        z = torch.polar(torch.full_like(s["freq"], s["amp"]).expand(at.numel(), -1).contiguous(), sign * at.double()[:, None] * s["freq"])[:, None]
        half = case["rot"] // 2
        even = torch.arange(0, case["rot"], 2, device="cuda") if case["inter"] else torch.arange(half, device="cuda")
        odd = even + (1 if case["inter"] else half)
        y = torch.complex(x[..., even], x[..., odd]) * z
        x = x.clone()
        x[..., even], x[..., odd] = y.real, y.imag
        return x

    if op == "rotate":
        at = s["positions"] if s["positions"] is not None else torch.cat([torch.arange(n, device="cuda") for n, _ in lens])
        return {name: turned(s[name], at, -1.0 if case["grad"] else 1.0) for name in ("q", "k")}
    layer = s["layers"][0]
    if op == "write":
        got = {"q": turned(s["q"], s["positions"], 1.0)}
        for name, x in (("k", turned(s["k"], s["positions"], 1.0)), ("v", s["v"].double())):
            pages = layer[name].double()
            scales = None if layer[name + "_scale"] is None else layer[name + "_scale"].double()
            if scales is not None:
                scale = torch.exp2(torch.clamp(torch.ceil(torch.log2(x.to(torch.bfloat16).double().abs().amax(-1) / E4M3_MAX)), min=-127.0))
                scales[s["slots"] // page, :, s["slots"] % page] = scale
                x = x / scale[..., None]
            pages[s["slots"] // page, s["slots"] % page] = x
            got[name], got[name + "_scale"] = pages, scales
        return got
    table, group = s["table"].tolist(), case["heads"] // case["kv_heads"]
    out = torch.zeros(s["total"], case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    lse = torch.full((case["heads"], s["total"]), -math.inf, dtype=torch.float64, device="cuda")
    above = torch.zeros(s["total"], max(n for n, _ in lens), dtype=torch.bool, device="cuda")
    parents = s["parents"].tolist()
    rows = [[] for _ in range(s["total"])]
    for b, (n, _) in enumerate(lens):  # each row's list is its parent's and itself
        for i in range(n):
            up = parents[cu[b] + i]
            rows[cu[b] + i] = (rows[cu[b] + up] if up >= 0 else []) + [i]
    at = torch.tensor([(r, i) for r, v in enumerate(rows) for i in v], device="cuda")
    above[at[:, 0], at[:, 1]] = True
    depth = above.sum(-1) - 1
    for b, (n, c) in enumerate(lens):
        j = torch.arange(n + c, device="cuda")
        of = torch.tensor(table[b], device="cuda")[j // page]

        def held(name):
            x = layer[name][of, j % page].double() if layer[name + "_scale"] is None else \
                layer[name].view(torch.uint8)[of, j % page].view(torch.float8_e4m3fn).double()
            return x if layer[name + "_scale"] is None else x * layer[name + "_scale"][of, :, j % page].double()[..., None]

        kk, vv = held("k"), held("v")
        mine = slice(cu[b], cu[b + 1])
        seen = torch.cat([torch.ones(n, c, dtype=torch.bool, device="cuda"), above[mine, :n]], 1)
        if case["left"] >= 0:
            seen[:, :c] &= j[:c] + case["left"] >= c + depth[mine, None]
        for h in range(case["heads"]):
            x = s["q"][mine, h].double() @ kk[:, h // group].T / math.sqrt(case["dim"])
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
            y = torch.logsumexp(x, -1)
            out[mine, h], lse[h, mine] = torch.exp(x - y[:, None]) @ vv[:, h // group], y
    return {"out": out, "lse": lse}
