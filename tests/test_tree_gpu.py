"""Attention of drafted trees over the cache, on a GPU, against a 64-bit form; and a step from the plan to the pages
given back, against the same tokens one after another."""
import math

import pytest
import torch

from tests import paged_cases as C
from tests import step_cases as S

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def va():
    from packed_variable_length_varlen_gb300 import varlen_attn
    return varlen_attn


def _ok(va):
    st = va.varlen_attn_get_device_status()
    assert st == 0, va.varlen_attn_status_string(st)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _tree(va, new, lens, heads, kv, dim, page, kind, left=-1, order="nhd", hint=None, seed=0, extra=0, pad=0, words=None,
          rows=None, garbage=False, columns=1, amp=1.0, shift=0, hide=0):
    """Runs and checks a call; rows: the lists of rows that each row sees (default: random trees); hide: new rows that
    nobody sees and that hold NaN."""
    g = torch.Generator().manual_seed(seed + 100)
    if rows is None:
        rows = [S.ancestors(S.random_tree(n, g)) for n in new]
    hidden = [set(torch.randperm(n, generator=g).tolist()[:hide]) if n > hide else set() for n in new]
    rows = [[[j for j in r if j not in h] for r in seq] for seq, h in zip(rows, hidden)]
    cache, k, v = C.make_cache(lens, kv, dim, page, kind, DEV, seed=seed, order=order, columns=columns, amp=amp)
    table = cache.block_table.tolist()
    for b, h in enumerate(hidden):
        for j in h:
            at = lens[b] - new[b] + j
            if at < 0:
                continue
            pg, r = table[b][at // page], at % page
            if kind == "bf16":
                cache.k_pages[pg, r], cache.v_pages[pg, r] = math.nan, math.inf
            else:
                cache.k_scale[pg, :, r], cache.v_scale[pg, :, r] = math.nan, math.nan
            k[b][at], v[b][at] = math.nan, math.nan
    total, words = sum(new) + extra, words or -(-max(max(new), 1) // 32)
    masks = torch.zeros(total, words, dtype=torch.int32)
    at = 0
    for n, seq in zip(new, rows):
        masks[at:at + n] = S.pack(seq, words)
        at += n
    if garbage:  # bits of rows that are not there
        at = 0
        for n in new:
            more = S.pack([range(n, 32 * words)], words)
            masks[at:at + n] |= more
            at += n
        masks[at:] = -1
    q = (torch.randn(total, heads, dim + pad, generator=g) * amp).to(torch.bfloat16).to(DEV)[..., :dim]
    depth = [max(len(r) - 1, 0) for seq in rows for r in seq]
    ctx = [lens[b] - n for b, n in enumerate(new) for _ in range(n)]
    pos = [c + d + shift for c, d in zip(ctx, depth)] + [0] * extra
    out = torch.full((total, heads, dim + pad), 77.0, dtype=torch.bfloat16, device=DEV)[..., :dim]
    lse = torch.full((heads, total), 77.0, device=DEV)
    call = lambda: va.attention_fwd_paged_tree(q, cache, C.cu_of(new, DEV), masks.to(DEV),  # noqa: E731
                                               max_seqlen_q=max(new) if hint is None else hint, window_left=left,
                                               positions=_ints(pos) if left >= 0 else None, out=out, lse=lse)
    call()
    _ok(va)
    scale = float(torch.tensor(dim ** -0.5, dtype=torch.float32))
    at = 0
    for b, n in enumerate(new):
        c = lens[b] - n
        seen = torch.zeros(n, lens[b], dtype=torch.bool)
        for i, r in enumerate(rows[b]):
            lo = max(0, max(pos[at + i], c) - left) if left >= 0 else 0
            if c > lo:
                seen[i, lo:c] = True
            for j in r:
                if c + j >= 0 and j < 32 * words:
                    seen[i, c + j] = True
        ref = S.attend_tree(q[at:at + n], k[b], v[b], scale, seen.to(DEV))
        C.check_attend(out[at:at + n], lse[:, at:at + n], ref, dim, lens[b])
        at += n
    assert (out[at:] == 77.0).all() and (lse[:, at:] == 77.0).all()  # rows behind the last segment stay
    first = (out.clone(), lse.clone())
    call()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])  # the same bits again
    return out, lse


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 2), (6, 1), (16, 2)])
def test_small_trees(va, kind, dim, heads, kv):
    """The kernel for few rows: up to 16 rows of a key head."""
    n = 16 // (heads // kv)
    _tree(va, [n, 1, 0, max(n - 1, 1), n], [200, 1, 40, 77, n], heads, kv, dim, 16, kind, extra=2, pad=32)
    _tree(va, [n, 1, 0, max(n - 1, 1), n], [200, 1, 40, 77, n], heads, kv, dim, 64, kind, order="hnd", left=20, garbage=True, words=2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("heads,kv,page", [(1, 1, 16), (4, 1, 64), (7, 1, 128), (24, 8, 32)])
def test_larger_trees(va, kind, dim, heads, kv, page):
    """The kernel for many rows, alone and beside the other one."""
    _tree(va, [64, 130, 0, 1, 300, 17], [500, 130, 33, 257, 300 + 128, 1000], heads, kv, dim, page, kind, extra=3, pad=32)
    _tree(va, [64, 130, 0, 1, 300, 17], [500, 130, 33, 257, 300 + 127, 1000], heads, kv, dim, page, kind, left=100, garbage=True, words=11, seed=4)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_both_kernels(va, kind):
    """Wide tables: small trees by one kernel, large ones by the other, in one call."""
    _tree(va, [150, 3, 4, 40], [900, 5000, 4, 41], 4, 2, 128, 64, kind, columns=1 << 14)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,hint", [([40], 3), ([3, 90, 5], 4), ([16, 200], 1)])
def test_a_hint_that_is_too_small(va, kind, new, hint):
    """The kernel for few rows takes trees of any size, 16 rows at a time."""
    _tree(va, new, [n + 100 for n in new], 4, 1, 128, 16, kind, hint=hint, hide=2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,lens", [([8, 2], [20000, 9000]), ([250], [30000]), ([64, 64], [9001, 17000])])
def test_trees_in_parts(va, kind, new, lens):
    """Long contexts, whose units several CTAs share."""
    _tree(va, new, lens, 4, 2, 64, 32, kind)
    _tree(va, new, lens, 4, 2, 64, 32, kind, left=5000, seed=2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,heads,kv,new,lens", [(64, 2, 1, [100], [60000]), (96, 6, 2, [40, 33], [30000, 1]), (128, 2, 1, [100], [60000]), (128, 5, 1, [60], [9000])])
def test_trees_in_many_parts(va, kind, dim, heads, kv, new, lens):
    """A few units over all SMs, in up to 17, 32 and more than 32 parts each; the causal band over the same cache."""
    lens = [max(n, m) for n, m in zip(lens, new)]
    _tree(va, new, lens, heads, kv, dim, 64, kind, extra=2)
    cache, k, v = C.make_cache(lens, kv, dim, 64, kind, DEV, seed=3)
    q = torch.randn(sum(new), heads, dim, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)
    out, lse = va.attention_fwd_paged(q, cache, C.cu_of(new, DEV), causal=True)
    _ok(va)
    at = 0
    for b, n in enumerate(new):
        seen = torch.arange(lens[b], device=DEV) <= torch.arange(lens[b] - n, lens[b], device=DEV)[:, None]
        ref = S.attend_tree(q[at:at + n], k[b], v[b], float(torch.tensor(dim ** -0.5, dtype=torch.float32)), seen)
        C.check_attend(out[at:at + n], lse[:, at:at + n], ref, dim, lens[b])
        at += n


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,kv,most,ctx,columns", [(8, 1, 40, 300, 1), (6, 2, 90, 700, 1), (16, 2, 12, 900, 1 << 13), (2, 2, 300, 2000, 1)])
def test_many_units(va, kind, heads, kv, most, ctx, columns):
    """Short and long units of one and of two halves, empty ones between them: wherever a CTA's part begins and ends."""
    g = torch.Generator().manual_seed(most)
    u = torch.rand(2, 48, generator=g).tolist()
    new = [0 if i % 7 == 3 else int(x * x * most) for i, x in enumerate(u[0])]
    lens = [n + int(x ** 3 * ctx) for n, x in zip(new, u[1])]
    _tree(va, new, lens, heads, kv, 64, 16, kind, columns=columns, extra=3)
    _tree(va, new, lens, heads, kv, 128, 32, kind, columns=columns, left=60, seed=1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,lens,heads", [([12], [100], 1), ([12, 5], [12, 300], 3), ([100], [180], 2), ([200, 70], [200, 500], 4), ([300], [1000], 1)])
def test_rows_that_nobody_sees(va, kind, new, lens, heads):
    """New rows outside every mask may hold NaN and infinities; rows whose mask is empty (and that have no context) give 0
    and -inf; a row need not see itself."""
    _tree(va, new, lens, heads, 1, 128, 16, kind, hide=5)
    _tree(va, new, lens, heads, 1, 96, 32, kind, hide=5, left=0, garbage=True)
    _tree(va, new, lens, heads, 1, 64, 32, kind, hide=3, left=60, shift=50)
    empty = [[[] if i % 3 == 0 else [max(i - 1, 0)] for i in range(n)] for n in new]
    _tree(va, new, lens, heads, 1, 128, 16, kind, rows=empty)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [2, 7, 40])
@pytest.mark.parametrize("left,shift", [(100, 60), (300, 290), (390, 200), (391, 390), (50, 70)])
def test_context_behind_every_window(va, kind, heads, left, shift):
    """Positions past the context: keys at the unit's start that no row sees, whole tiles of them too, hold NaN."""
    new, lens = [9], [400]
    cache, k, v = C.make_cache(lens, 1, 128, 16, kind, DEV)
    c = 391  # rows see [c + shift - left, c)
    shown = min(shift, left)
    table = cache.block_table[0].tolist()
    for at in range(c - left, c + shown - left):
        pg, r = table[at // 16], at % 16
        if kind == "bf16":
            cache.k_pages[pg, r], cache.v_pages[pg, r] = math.nan, math.nan
        else:
            cache.k_scale[pg, :, r], cache.v_scale[pg, :, r] = math.nan, math.nan
        k[0][at], v[0][at] = 0, 0
    q = torch.randn(9, heads, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    masks = S.pack([[i] for i in range(9)], 1).to(DEV)
    out, lse = va.attention_fwd_paged_tree(q, cache, C.cu_of(new, DEV), masks, max_seqlen_q=9, window_left=left,
                                           positions=_ints([c + shift] * 9))
    _ok(va)
    seen = torch.zeros(9, 400, dtype=torch.bool, device=DEV)
    seen[:, c + shown - left:c] = True
    seen[torch.arange(9), c + torch.arange(9)] = True
    C.check_attend(out, lse, S.attend_tree(q, k[0], v[0], float(torch.tensor(128 ** -0.5)), seen), 128, 400)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_more_rows_than_positions(va, kind):
    """A sequence that holds fewer positions than rows came: the first rows have no place and nobody sees them."""
    _tree(va, [20, 9], [15, 0], 2, 1, 64, 16, kind)
    _tree(va, [90, 9], [70, 3], 4, 1, 128, 16, kind, left=30)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,lens,heads", [(7, 300, 2), (60, 300, 8), (200, 200, 1)])
def test_a_chain_is_causal(va, kind, n, lens, heads):
    """Masks of a chain give what the band gives: the same kernels, whose CTAs share the tiles out in another way."""
    cache, _, _ = C.make_cache([lens], 1, 128, 16, kind, DEV)
    q = torch.randn(n, heads, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    masks = S.pack([range(i + 1) for i in range(n)], -(-n // 32)).to(DEV)
    cu = C.cu_of([n], DEV)
    a = va.attention_fwd_paged_tree(q, cache, cu, masks, max_seqlen_q=n)
    b = va.attention_fwd_paged(q, cache, cu, max_seqlen_q=n, causal=True)
    _ok(va)
    ref = S.attend_tree(q, *_held(va, cache, lens), 128 ** -0.5, torch.arange(lens, device=DEV) <= torch.arange(lens - n, lens, device=DEV)[:, None])
    C.check_attend(a[0], a[1], ref, 128, lens)
    # two orders of the same sums, each within the bounds of check_attend
    tol = 2 * (2.0 ** -8 * (ref[2] + ref[0].abs()) + 2.0 ** -14 * ref[2])
    assert ((a[0].double() - b[0].double()).abs() <= tol).all()


def _held(va, cache, n):
    k, v = va.cache_read(cache, C.cu_of([n], DEV), n)
    return k.double(), v.double()


# loads of CTA 0, K and V counted alike: 5000 keys are 79 tiles of 64 and 40 of 128, so CTA 0 has at least 2 tiles
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("which,new,columns", [(3, [3, 2], 1), (4, [100, 3], 1), (4, [70, 1], 1 << 14)])
@pytest.mark.parametrize("load", [0, 3])
def test_a_skipped_load_times_out_and_the_next_call_is_right(va, kind, which, new, columns, load):
    """3: the kernel for few rows, 4: the one for many; the bounded waits run out, the call says so, the context lives on."""
    assert va.varlen_attn_get_device_status() == 0
    # (330 tiles in the kernel for many rows: two of them at least in every CTA, the first one's too)
    cache, _, _ = C.make_cache([20000, 900], 2, 128, 64, kind, DEV, columns=columns)
    q = torch.randn(sum(new), 4, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    masks = torch.full((sum(new), 4), -1, dtype=torch.int32, device=DEV)
    assert va.varlen_attn_debug_skip_load(which, load) == 0
    try:
        va.attention_fwd_paged_tree(q, cache, C.cu_of(new, DEV), masks, max_seqlen_q=max(new))
        st = va.varlen_attn_get_device_status()
    finally:
        va.varlen_attn_debug_skip_load(which, -1)
    assert st == va.VARLEN_ERR_TIMEOUT, va.varlen_attn_status_string(st)
    _tree(va, new, [5000, 900], 4, 2, 128, 64, kind, columns=columns)


def test_other_streams(va):
    """On another stream than the current one: every operator's result is the same, memory that a call allocates included."""
    kind, new, lens = "e4m3", [20, 3], [300, 77]
    cache, _, _ = C.make_cache(lens, 2, 64, 16, kind, DEV)
    q = torch.randn(23, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    k = q[:, :2].contiguous()
    masks = torch.cat([S.pack(S.ancestors(S.random_tree(n, torch.Generator().manual_seed(n))), 1) for n in new]).to(DEV)
    rope = va.Rotary(va.rotary_frequencies(64)[0], device=DEV)
    pos, slots = _ints(list(range(23))), _ints(list(range(23)), torch.int64)
    side = torch.cuda.Stream()

    def all_of_it(stream):
        torch.cuda._sleep(2000000)  # what the current stream still does with recycled memory
        junk = [torch.full((23, 4, 64), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
        del junk
        a, b = va.rotary(q, k, rope, positions=pos, stream=stream)
        c = va.rotary_cache_write(cache, q, k, k, rope, pos, slots, stream=stream)
        out, lse = va.attention_fwd_paged_tree(c, cache, C.cu_of(new, DEV), masks, max_seqlen_q=20, stream=stream)
        pool = va.PagePool(cache.block_table.clone(), _ints([5, 0]), torch.arange(30, dtype=torch.int32, device=DEV), _ints([30]), 16)
        plan = va.StepPlan(2, 30, DEV, mask_words=1)
        torch.cuda.synchronize()
        va.cache_plan(pool, plan, _ints(new), parents=torch.full((30,), -1, dtype=torch.int32, device=DEV), stream=None)
        torch.cuda.synchronize()
        va.cache_move(cache, plan.cu_seqlens, _ints([[2, 5], [1, 2]]), _ints([2, 2]), stream=stream)
        va.cache_trim(pool, _ints([1, 1]), plan.cu_seqlens, stream=stream)
        torch.cuda.synchronize()
        return [a, b, c, out, lse, pool.seqlens, pool.free_pages, pool.free_count, plan.slots, plan.masks, cache.k_pages.view(torch.uint8).clone()]

    ref = all_of_it(None)
    for stream in (side, side.cuda_stream):
        cache2, _, _ = C.make_cache(lens, 2, 64, 16, kind, DEV)
        for x, y in zip((cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale), (cache2.k_pages, cache2.v_pages, cache2.k_scale, cache2.v_scale)):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        for x, y in zip(all_of_it(stream), ref):
            assert torch.equal(x, y)
    _ok(va)


# ------------------------------------------------------------------ a step, whole

class _Model:
    """Layers of projections around the attention, for tokens that a table gives."""

    def __init__(self, va, kind, layers=2, heads=4, kv=2, dim=64, vocab=50):
        g = torch.Generator().manual_seed(7)
        self.va, self.kind, self.heads, self.kv, self.dim, self.layers = va, kind, heads, kv, dim, layers
        self.embed = torch.randn(vocab, heads * dim, generator=g).to(DEV)
        self.w = [[(torch.randn(heads * dim, n * dim, generator=g) * (heads * dim) ** -0.5).to(DEV) for n in (heads, kv, kv)]
                  for _ in range(layers)]
        self.rope = va.Rotary(va.rotary_frequencies(dim)[0], device=DEV)

    def caches(self, table, seqlens, pages, page):
        dt = torch.bfloat16 if self.kind == "bf16" else torch.float8_e4m3fn
        got = []
        for _ in range(self.layers):
            p = [torch.zeros(pages, page, self.kv, self.dim, device=DEV).to(dt) for _ in range(2)]
            s = [None if self.kind == "bf16" else torch.ones(pages, self.kv, page, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            got.append(self.va.PagedCache(*p, table, seqlens, *s))
        return got

    def step(self, caches, plan, tokens, most, tree):
        x = self.embed[tokens]
        for cache, (wq, wk, wv) in zip(caches, self.w):
            h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
            q, k, v = ((h @ w).to(torch.bfloat16).unflatten(1, (-1, self.dim)) for w in (wq, wk, wv))
            q = self.va.rotary_cache_write(cache, q, k, v, self.rope, plan.positions, plan.slots)
            if tree:
                o, _ = self.va.attention_fwd_paged_tree(q, cache, plan.cu_seqlens, plan.masks, max_seqlen_q=most)
            else:
                o, _ = self.va.attention_fwd_paged(q, cache, plan.cu_seqlens, max_seqlen_q=most, causal=True)
            x = x + o.flatten(1).float()
        return x


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("graph", [False, True])
def test_a_step_from_plan_to_trim(va, kind, graph):
    """Prompts, then drafted trees, the accepted paths kept, then one more token: as the same tokens fed one path at a
    time into a cache of their own.  What a token's row holds does not depend on the tree around it; sums in another
    order move O by bf16's last bits, layer by layer, which 2% of the largest value covers many times."""
    m = _Model(va, kind)
    prompts, page, width, pages = [37, 5, 130], 16, 20, 70
    trees = [[-1, 0, 0, 1, 1, 2, 3, 6], [-1, -1, 1, 2, 0], [-1] + list(range(20))]
    paths = [[0, 1, 3, 6, 7], [1, 2], [0, 1, 2, 3]]
    g = torch.Generator().manual_seed(1)
    tok = [torch.randint(0, 50, (n,), generator=g).to(DEV) for n in prompts]
    draft = [torch.randint(0, 50, (len(t),), generator=g).to(DEV) for t in trees]
    after = torch.randint(0, 50, (3,), generator=g).to(DEV)

    def fresh():
        table = torch.zeros(3, width, dtype=torch.int32, device=DEV)
        seqlens = _ints([0] * 3)
        pool = va.PagePool(table, seqlens, torch.randperm(pages, generator=g).to(torch.int32).to(DEV), _ints([pages]), page)
        return pool, m.caches(table, seqlens, pages, page)

    pool, caches = fresh()
    plan = va.StepPlan(3, sum(prompts), DEV)
    m.step(caches, va.cache_plan(pool, plan, _ints(prompts)), torch.cat(tok), max(prompts), False)
    room = sum(len(t) for t in trees) + 6  # a padded step
    plan = va.StepPlan(3, room, DEV, mask_words=1)
    lens, parents = _ints([0] * 3), _ints([0] * room)
    tokens = torch.zeros(room, dtype=torch.long, device=DEV)
    kept, kept_lens = torch.zeros(3, 6, dtype=torch.int32, device=DEV), _ints([0] * 3)
    x = torch.zeros(room, 256, device=DEV)

    def whole():
        va.cache_plan(pool, plan, lens, parents=parents)
        x.copy_(m.step(caches, plan, tokens, 32, True))
        va.cache_move(caches, plan.cu_seqlens, kept, kept_lens)
        va.cache_trim(pool, kept_lens, plan.cu_seqlens)

    if graph:  # captured on empty steps, replayed on real ones
        whole()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            whole()
        torch.cuda.current_stream().wait_stream(side)
        replay = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replay):
            whole()
    lens.copy_(_ints([len(t) for t in trees]))
    parents[:room - 6] = _ints(sum(trees, []))
    tokens[:room - 6] = torch.cat(draft)
    for b, p in enumerate(paths):
        kept[b, :len(p)] = _ints(p)
    kept_lens.copy_(_ints([len(p) for p in paths]))
    replay.replay() if graph else whole()
    _ok(va)
    assert pool.seqlens.tolist() == [n + len(p) for n, p in zip(prompts, paths)]
    assert pool.free_count.item() == pages - sum(-(-n // page) for n in pool.seqlens.tolist())
    owned = [pool.block_table[b, :-(-n // page)].tolist() for b, n in enumerate(pool.seqlens.tolist())]
    assert sorted(sum(owned, []) + pool.free_pages[:pool.free_count.item()].tolist()) == list(range(pages))
    plan1 = va.StepPlan(3, 3, DEV)
    y = m.step(caches, va.cache_plan(pool, plan1, _ints([1, 1, 1])), after, 1, False)
    _ok(va)

    # every path of every tree by itself
    at = 0
    for b, t in enumerate(trees):
        rows = S.ancestors(t)
        for i, r in enumerate(rows):
            if i % 3 != 2 and r != paths[b]:
                continue
            p2, c2 = fresh()
            one = lambda n: _ints([n if s == b else 0 for s in range(3)])  # noqa: E731
            pl = va.cache_plan(p2, va.StepPlan(3, prompts[b], DEV), one(prompts[b]))
            m.step(c2, pl, tok[b], prompts[b], False)
            pl = va.cache_plan(p2, va.StepPlan(3, len(r), DEV), one(len(r)))
            z = m.step(c2, pl, draft[b][torch.tensor(r, device=DEV)], len(r), False)
            assert (z[-1] - x[at + i]).abs().max() <= 0.02 * z.abs().max()
            if r == paths[b]:
                pl = va.cache_plan(p2, va.StepPlan(3, 1, DEV), one(1))
                z = m.step(c2, pl, after[b:b + 1], 1, False)
                assert (z[0] - y[b]).abs().max() <= 0.02 * z.abs().max()
        at += len(t)
    _ok(va)
