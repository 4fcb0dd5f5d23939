"""Cases of the paged key/value cache and the attention that reads it.

Three operators over one cache, in bf16 and in E4M3:

* ``write``  -- new keys and values, packed by cu_seqlens, go to their places
  in the pages (E4M3: one power-of-two scale for each token and head);
* ``read``   -- the last rows of every sequence come back, packed, in bf16;
* ``attend`` -- packed new queries over the pages, query heads sharing key
  heads, under the band of the packed forward (diagonal at the last key):
  single tokens, a few drafted ones, chunks of a prompt, and mixtures.

``own`` chooses between a plain form in elementary torch operations and the
library's entry points.  A case gives the ranges of its lengths and a number
``shape`` that they are drawn from; values and page order come from the seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _case(name, op, kind, shape, seqs, new, ctx, heads, kv_heads, dim, page, causal=True, left=-1, ones=0):
    return {"name": name, "op": op, "type": kind, "shape": shape, "seqs": seqs, "new_lo": new[0], "new_hi": new[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "causal": causal, "left": left, "ones": ones}


def listed():
    return [
        # the cache update of one decoding step of a small batch: latency
        _case("write_tokens_e4m3", "write", "e4m3", 1, 16, (1, 1), (1, 2000), 32, 8, 128, 16),
        # the ragged workload's prompts (64 sequences of up to 8192 rows) into an empty cache
        _case("write_prompts_e4m3", "write", "e4m3", 2, 64, (0, 8192), (0, 0), 32, 32, 128, 64),
        # two long prompts of head size 96 into a bf16 cache
        _case("write_prompts_bf16", "write", "bf16", 3, 2, (9001, 20011), (0, 0), 16, 16, 96, 32),
        # the windowed workload's keys (8 windows of 17580 rows, 56 heads) read back for a packed call
        _case("read_context_e4m3", "read", "e4m3", 4, 8, (17580, 17580), (17580, 17580), 56, 56, 128, 16),
        # a few short prefixes read back: latency
        _case("read_prefix_bf16", "read", "bf16", 5, 4, (37, 500), (0, 600), 2, 2, 64, 16),
        # four drafted tokens of a few sequences verified under a sliding window: latency
        _case("draft_window_bf16", "attend", "bf16", 6, 4, (4, 4), (500, 4000), 16, 4, 64, 16, left=1023),
        # one decoding step of a full batch at ragged lengths
        _case("decode_batch_e4m3", "attend", "e4m3", 7, 64, (1, 1), (1, 8192), 32, 8, 128, 64),
        # one decoding step where every query head has its own keys (the windowed workload's heads and keys)
        _case("decode_heads_bf16", "attend", "bf16", 8, 8, (1, 1), (17580, 17580), 56, 56, 128, 128),
        # one decoding step of one very long sequence (the strided workload's length, heads and head size)
        _case("decode_long_e4m3", "attend", "e4m3", 9, 1, (1, 1), (185619, 185619), 16, 2, 96, 256),
        # chunks of four prompts over what came before
        _case("chunk_bf16", "attend", "bf16", 10, 4, (1500, 2048), (4096, 16384), 32, 8, 128, 64),
        # one step of a server: most sequences decode, two bring a chunk
        _case("mixed_e4m3", "attend", "e4m3", 11, 16, (300, 512), (100, 8192), 32, 8, 128, 16, ones=14),
        # a short chunk at the end of the long workload: few rows, 77000 keys, seven query heads to a key head
        _case("chunk_long_e4m3", "attend", "e4m3", 12, 1, (250, 250), (77000, 77000), 56, 8, 128, 64),
    ]


def _lens(case):
    """[(new rows, rows in the cache with them)] of every sequence."""
    r = random.Random(1000 + case["shape"])
    got = []
    for b in range(case["seqs"]):
        new = 1 if b < case["ones"] else r.randint(case["new_lo"], case["new_hi"])
        got.append((new, max(new, r.randint(case["ctx_lo"], case["ctx_hi"]))))
    r.shuffle(got)
    return got


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "attend"))
    kind = rng.choice(("bf16", "e4m3"))
    while True:
        seqs = _spread(rng, 1, 64)
        hi = _spread(rng, 16, 77000)
        kv = rng.choice((1, 2, 3, 4, 8, 16, 32, 56))
        group = rng.choice((1, 2, 3, 4, 5, 7, 8, 16)) if op == "attend" else 1
        form = rng.choice(("token", "draft", "chunk", "mixed")) if op == "attend" else rng.choice(("token", "chunk"))
        new_hi = {"token": 1, "draft": rng.randint(2, 9)}.get(form) or min(hi, _spread(rng, 16, 2048 if op == "attend" else 8192))
        case = _case("", op, kind, rng.randrange(1 << 20), seqs, (1 if form == "token" else rng.randint(1, new_hi), new_hi),
                     (rng.randint(0, hi), hi), kv * group, kv, rng.choice((64, 96, 128)), rng.choice((16, 32, 64, 128, 256)),
                     rng.random() < 0.8, rng.choice((-1, -1, -1, _spread(rng, 1, 8192))), rng.randint(0, seqs) if form == "mixed" else 0)
        del case["name"]
        w = work(case)
        if kv * group <= 64 and w["bytes"] <= 4e9 and w["flops"] <= 1.2e12 and _padded(case) <= 2.5e9:
            return case


def _padded(case):
    """Entries of the plain form's score tensor."""
    lens = _lens(case)
    return case["seqs"] * case["heads"] * max(n for n, _ in lens) * max(1, max(k for _, k in lens)) if case["op"] == "attend" else 0


def _right(case):
    return 0 if case["causal"] else -1


def _row_bytes(case):
    """Bytes of one row of one key head in the cache: K or V."""
    return case["dim"] * 2 if case["type"] == "bf16" else case["dim"] + 2


def work(case):
    lens, kv, dim = _lens(case), case["kv_heads"], case["dim"]
    rows = sum(n for n, _ in lens)
    if case["op"] != "attend":
        return {"bytes": 2 * rows * kv * (2 * dim + _row_bytes(case)), "flops": 0}
    keys = pairs = 0
    for n, k in lens:
        left, right = case["left"], _right(case)
        first = max(0, k - n - left) if left >= 0 else 0
        keys += k - first if n else 0
        for i in range(n):
            lo = max(0, k - n + i - left) if left >= 0 else 0
            pairs += (min(k, k - n + i + right + 1) if right >= 0 else k) - lo
    return {"bytes": 2 * keys * kv * _row_bytes(case) + rows * case["heads"] * (4 * dim + 4), "flops": 4 * pairs * case["heads"] * dim}


# ------------------------------------------------------------------ inputs

def _hold(x):
    """(codes as their values, scale) of rows x [..., dim] in 32 bits: scale the least power of two with
    amax <= 448 * scale (1 for rows of zeros), code = x / scale rounded to E4M3."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.clamp(e - 9 + (m > 0.875), min=-127)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    return torch.clamp(x / scale[..., None], -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    lens, kv, dim, page = _lens(case), case["kv_heads"], case["dim"], case["page"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    need = [-(-k // page) for _, k in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [0] * (max(need) - n))
        at += n
    s = {"case": case, "total": sum(n for n, _ in lens), "max_new": max(n for n, _ in lens), "max_keys": max(k for _, k in lens)}
    s["cu"] = torch.tensor([0] + [n for n, _ in lens], dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)
    s["seqlens"] = torch.tensor([k for _, k in lens], dtype=torch.int32, device="cuda")
    s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda").reshape(len(lens), max(need))
    shape = (pages, page, kv, dim)
    empty = case["op"] == "write"
    for name in ("k", "v"):
        x = torch.zeros(shape, device="cuda") if empty else normal(*shape)
        if case["type"] == "bf16":
            s[name + "_pages"], s[name + "_scale"] = x.to(torch.bfloat16), None
        else:
            # heads and tokens differ in size, as keys and values do
            size = torch.exp2(torch.randint(-3, 3, shape[:3], generator=g, device="cuda").float())
            codes, scale = _hold((x * size[..., None]).to(torch.bfloat16).float())
            s[name + "_pages"], s[name + "_scale"] = codes, scale.transpose(1, 2).contiguous()
        del x
        if empty:
            s[name + "_new"] = normal(s["total"], kv, dim).to(torch.bfloat16)
    if case["op"] == "attend":
        s["q"] = normal(s["total"], case["heads"], dim).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ the plain form

def _places(s):
    """(page, row) in the cache of every packed row: the last rows of its sequence."""
    row = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    at = row - s["cu"][b + 1] + s["seqlens"][b]
    return s["table"][b, at // s["case"]["page"]].long(), at % s["case"]["page"]


def _write(s, name):
    page, row = _places(s)
    pages, scales = s[name + "_pages"], s[name + "_scale"]
    if scales is None:
        pages[page, row] = s[name + "_new"]
    else:
        codes, scale = _hold(s[name + "_new"].float())
        pages.view(torch.uint8)[page, row] = codes.view(torch.uint8)
        scales[page, :, row] = scale
    return pages, scales


def _values(s, name, page, row):
    """Cache rows [..., kv heads, dim] in 32 bits."""
    pages, scales = s[name + "_pages"], s[name + "_scale"]
    if scales is None:
        return pages[page, row].float()
    return pages.view(torch.uint8)[page, row].view(torch.float8_e4m3fn).float() * scales.transpose(1, 2)[page, row].float()[..., None]


def _attend(s):
    case, group = s["case"], s["case"]["heads"] // s["case"]["kv_heads"]
    t, j = torch.arange(s["max_new"], device="cuda"), torch.arange(s["max_keys"], device="cuda")
    new, keys = (s["cu"][1:] - s["cu"][:-1]).long(), s["seqlens"].long()
    inside = t[None] < new[:, None]
    packed = (s["cu"][:-1].long()[:, None] + t[None])[inside]
    # queries [seqs, kv heads, rows * group, dim]
    q = torch.zeros(case["seqs"], s["max_new"], case["heads"], case["dim"], device="cuda")
    q[inside] = s["q"][packed].float()
    q = q.unflatten(2, (case["kv_heads"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    page, row = s["table"][:, j // case["page"]].long(), (j % case["page"]).expand(case["seqs"], -1)
    x = (q @ _values(s, "k", page, row).permute(0, 2, 3, 1)) * (1.0 / math.sqrt(case["dim"]))
    at = t[None] + (keys - new)[:, None]  # the last key stands at the last query
    seen = (j[None, None] < keys[:, None, None]).expand(-1, s["max_new"], -1)
    if case["causal"]:
        seen = seen & (j[None, None] <= at[..., None])
    if case["left"] >= 0:
        seen = seen & (j[None, None] >= at[..., None] - case["left"])
    x.masked_fill_(~seen.repeat_interleave(group, 1)[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x @ _values(s, "v", page, row).transpose(1, 2)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + total.log()

    def back(y):  # [seqs, kv heads, rows * group, n] -> [packed rows, heads, n]
        return y.unflatten(2, (s["max_new"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)[inside]

    return back(out).to(torch.bfloat16), back(lse)[..., 0].T.contiguous()


def run(s):
    op = s["case"]["op"]
    if own:
        from packed_variable_length_varlen_gb300 import varlen_attn as va
        if "cache" not in s:  # the handle that a program keeps beside its pages
            s["cache"] = va.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["seqlens"], s["k_scale"], s["v_scale"])
        if op == "write":
            va.cache_write(s["cache"], s["k_new"], s["v_new"], s["cu"])
            return {"k": s["k_pages"], "v": s["v_pages"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        if op == "read":
            k, v = va.cache_read(s["cache"], s["cu"], s["total"])
            return {"k": k, "v": v}
        out, lse = va.attention_fwd_paged(s["q"], s["cache"], s["cu"], max_seqlen_q=s["max_new"], causal=s["case"]["causal"],
                                          window=(s["case"]["left"], -1))
        return {"out": out, "lse": lse}
    if op == "write":
        (k, ks), (v, vs) = _write(s, "k"), _write(s, "v")
        return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}
    if op == "read":
        page, row = _places(s)
        return {"k": _values(s, "k", page, row).to(torch.bfloat16), "v": _values(s, "v", page, row).to(torch.bfloat16)}
    out, lse = _attend(s)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    lens, page = _lens(case), case["page"]
    table, cu = s["table"].tolist(), s["cu"].tolist()
    group = case["heads"] // case["kv_heads"]

    def held(name, b, first, last):
        """Rows [first, last) of sequence b: [rows, kv heads, dim]."""
        at = torch.arange(first, last, device="cuda")
        of = torch.tensor(table[b] or [0], device="cuda")[at // page]
        x = s[name + "_pages"][of, at % page].double() if s[name + "_scale"] is None else \
            s[name + "_pages"].view(torch.uint8)[of, at % page].view(torch.float8_e4m3fn).double()
        return x if s[name + "_scale"] is None else x * s[name + "_scale"][of, :, at % page].double()[..., None]

    if case["op"] == "write":
        got = {}
        for name in ("k", "v"):
            pages = s[name + "_pages"].double()
            scales = None if s[name + "_scale"] is None else s[name + "_scale"].double()
            for b, (n, k) in enumerate(lens):
                at = torch.arange(k - n, k, device="cuda")
                of = torch.tensor(table[b] or [0], device="cuda")[at // page]
                x = s[name + "_new"][cu[b]:cu[b + 1]].double()
                if scales is not None:
                    amax = x.abs().amax(-1)
                    scale = torch.exp2(torch.clamp(torch.ceil(torch.log2(amax / E4M3_MAX)), min=-127.0))
                    scale = torch.where(amax > 0, scale, torch.ones_like(scale))
                    scales[of, :, at % page] = scale
                    x = x / scale[..., None]
                pages[of, at % page] = x
            got[name], got[name + "_scale"] = pages, scales
        return got
    if case["op"] == "read":
        return {name: torch.cat([held(name, b, k - n, k) for b, (n, k) in enumerate(lens)]) for name in ("k", "v")}
    out = torch.zeros(s["total"], case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    lse = torch.full((case["heads"], s["total"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, k) in enumerate(lens):
        if n == 0 or k == 0:
            continue
        kk, vv = held("k", b, 0, k), held("v", b, 0, k)
        at, j = torch.arange(k - n, k, device="cuda")[:, None], torch.arange(k, device="cuda")[None]
        seen = torch.ones(n, k, dtype=torch.bool, device="cuda")
        if case["causal"]:
            seen &= j <= at
        if case["left"] >= 0:
            seen &= j + case["left"] >= at
        for h in range(case["heads"]):
            x = s["q"][cu[b]:cu[b + 1], h].double() @ kk[:, h // group].T / math.sqrt(case["dim"])
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
            y = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(torch.isfinite(y), y, torch.zeros_like(y))[:, None])
            out[cu[b]:cu[b + 1], h], lse[h, cu[b]:cu[b + 1]] = p @ vv[:, h // group], y
    return {"out": out, "lse": lse}
