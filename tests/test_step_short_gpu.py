"""Steps whose sequences run past their tables, on a GPU: the rows that have a place are written, attended, moved and
given back as those of any other sequence, from the plan to the trim, against a 64-bit form over what the cache holds."""
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


def _ok(va, want=0):
    st = va.varlen_attn_get_device_status()
    assert st == want, va.varlen_attn_status_string(st)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class _Step:
    """A plan over sequences that hold random rows, its new rows written and attended."""

    def __init__(self, va, kind, old, new, width, page, heads, kv, dim, free=8, extra=2, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.va, self.kind, self.old, self.new, self.width, self.page, self.dim = va, kind, old, new, width, page, dim
        need = [-(-n // page) for n in old]
        names = torch.randperm(sum(need) + free, generator=g).tolist()
        self.pages, at, table = len(names), 0, []
        for n in need:
            table.append(names[at:at + n] + [-9] * (width - n))
            at += n
        self.stack = names[at:]
        self.table, self.seqlens = _ints(table), _ints(old)
        free_pages = _ints(self.stack + [-9] * at)
        self.pool = va.PagePool(self.table, self.seqlens, free_pages, _ints([free]), page)
        x = [torch.randn(self.pages, page, kv, dim, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
        scales = [None, None]
        if kind == "e4m3":
            codes = [C.quantise(t) for t in x]
            x, scales = [c for c, _ in codes], [s.transpose(1, 2).contiguous() for _, s in codes]
        self.cache = va.PagedCache(*x, self.table, self.seqlens, *scales)
        total = sum(new) + extra
        words = -(-max(new) // 32)
        self.trees = [S.random_tree(n, g) for n in new]
        self.plan = va.StepPlan(len(old), total, DEV, mask_words=words)
        va.cache_plan(self.pool, self.plan, _ints(new), parents=_ints(sum(self.trees, []) + [-1] * extra))
        rope = va.Rotary(va.rotary_frequencies(dim)[0], device=DEV)
        q, k, v = (torch.randn(total, h, dim, generator=g).to(torch.bfloat16).to(DEV) for h in (heads, kv, kv))
        self.q = va.rotary_cache_write(self.cache, q, k, v, rope, self.plan.positions, self.plan.slots)

    def pools(self):
        got = [self.cache.k_pages.view(torch.uint8).clone(), self.cache.v_pages.view(torch.uint8).clone()]
        return got + [s.clone() for s in (self.cache.k_scale, self.cache.v_scale) if s is not None]

    def held(self, b):
        """What the cache's calls read of sequence b's table: positions without a page are zeros."""
        got = []
        for t, s in ((self.cache.k_pages, self.cache.k_scale), (self.cache.v_pages, self.cache.v_scale)):
            x = t.double() if s is None else t.double() * s.transpose(1, 2).double()[..., None]
            rows = [x[p] if 0 <= p < self.pages else torch.zeros_like(x[0]) for p in self.table[b].tolist()]
            got.append(torch.cat(rows))
        return got

    def place(self, b, at):
        p = self.table[b, at // self.page].item() if at < self.width * self.page else -1
        return p if 0 <= p < self.pages else -1

    def attend(self, left=-1):
        va, cap = self.va, self.width * self.page
        out, lse = va.attention_fwd_paged_tree(self.q, self.cache, self.plan.cu_seqlens, self.plan.masks, max_seqlen_q=max(self.new),
                                               window_left=left, positions=self.plan.positions if left >= 0 else None)
        scale, at = float(torch.tensor(self.dim ** -0.5, dtype=torch.float32)), 0
        for b, n in enumerate(self.new):
            ctx, rows = self.old[b], S.ancestors(self.trees[b])
            held = min(ctx + n, cap)
            seen = torch.zeros(n, cap, dtype=torch.bool)
            for i, r in enumerate(rows):
                lo = max(0, ctx + len(r) - 1 - left) if left >= 0 else 0
                seen[i, lo:max(min(ctx, cap), lo)] = True
                for j in r:
                    if ctx + j < cap:
                        seen[i, ctx + j] = True
            ref = S.attend_tree(self.q[at:at + n], *self.held(b), scale, seen.to(DEV))
            C.check_attend(out[at:at + n], lse[:, at:at + n], ref, self.dim, held)
            at += n

    def keep(self, kept):
        """cache_move and cache_trim, checked; kept: lists of accepted rows."""
        va, want = self.va, self.pools()
        before = [p.clone() for p in want]
        for b, rows in enumerate(kept):
            for i, r in enumerate(rows):
                (src, f), (dst, t) = ((self.place(b, x), x % self.page) for x in (self.old[b] + r, self.old[b] + i))
                if src < 0 or dst < 0:
                    continue
                for n, p in enumerate(want):
                    if n < 2:
                        p[dst, t] = before[n][src, f]
                    else:
                        p[dst, :, t] = before[n][src, :, f]
        most = max(len(r) for r in kept)
        va.cache_move(self.cache, self.plan.cu_seqlens, _ints([r + [0] * (most - len(r)) for r in kept]), _ints([len(r) for r in kept]))
        for x, y in zip(self.pools(), want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        table = self.table.tolist()
        va.cache_trim(self.pool, _ints([len(r) for r in kept]), self.plan.cu_seqlens)
        cap = self.width * self.page
        stay = [min(o + len(r), cap) for o, r in zip(self.old, kept)]
        assert self.seqlens.tolist() == stay
        own = [p for b, n in enumerate(stay) for p in table[b][:-(-n // self.page)] if p >= 0]
        free = self.pool.free_pages[:self.pool.free_count.item()].tolist()
        assert sorted(own + free) == list(range(self.pages))


# (positions before the step, new rows, table's width, page): the first sequence's rows end past its table
PAST = [(79, 2, 5, 16), (70, 14, 5, 16), (70, 40, 5, 16), (80, 3, 5, 16), (65, 40, 5, 16), (170, 9, 11, 16), (175, 90, 11, 16), (380, 30, 12, 32),
        (384, 70, 12, 32), (257, 200, 9, 32)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,kv", [(2, 2), (7, 1), (8, 2)])
@pytest.mark.parametrize("old,n,width,page", PAST)
def test_a_sequence_past_its_table(va, kind, heads, kv, old, n, width, page):
    """Its rows stand behind its own context, wherever the table ends: those that have a place see it and one another."""
    s = _Step(va, kind, [old, 20, 0], [n, 7, 5], width, page, heads, kv, 64)
    lost = old + n - width * page
    assert lost > 0 and s.plan.unplaced.tolist() == [lost, 0, 0] and s.seqlens.tolist() == [old + n, 27, 5]
    s.attend()
    for left in (0, 9, 60):
        s.attend(left)
    _ok(va)
    placed = max(n - lost, 0)
    s.keep([sorted({0, placed - 1, placed // 2}) if placed > 0 else [], [0, 3], [1, 2, 4]])
    _ok(va)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [1, 32])
@pytest.mark.parametrize("length", [81, 200, 2 ** 31 - 1])
def test_lengths_past_the_table(va, kind, heads, length):
    """However far: rows past the table have no keys of their own, and see all of a context that fills it."""
    cache, k, v = C.make_cache([80, 30], 1, 128, 16, kind, DEV)
    cache.seqlens[0] = length
    new = [2, 3]
    q = torch.randn(5, heads, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    masks = torch.full((5, 1), -1, dtype=torch.int32, device=DEV)
    out, lse = va.attention_fwd_paged_tree(q, cache, C.cu_of(new, DEV), masks, max_seqlen_q=3)
    _ok(va)
    for b, (lo, hi, keys) in enumerate(((0, 2, 80), (2, 5, 30))):
        seen = torch.ones(hi - lo, keys, dtype=torch.bool, device=DEV)
        ref = S.attend_tree(q[lo:hi], k[b], v[b], float(torch.tensor(128 ** -0.5, dtype=torch.float32)), seen)
        C.check_attend(out[lo:hi], lse[:, lo:hi], ref, 128, keys)


# ------------------------------------------------------------------ too few pages

SHORT = [
    # (positions before the step, new rows, table's width, page, free pages): who gets none, from the first whose running need
    # is above them on (the others that need none keep all their rows)
    ([10, 60, 14, 33, 30], [7, 40, 5, 4, 9], 8, 16, 2),
    ([0, 100, 5], [3, 60, 2], 12, 16, 0),
    ([130, 7, 250], [200, 9, 60], 16, 32, 4),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 2)])
@pytest.mark.parametrize("old,new,width,page,free", SHORT)
def test_a_step_short_of_pages(va, kind, heads, kv, old, new, width, page, free):
    """Sequences that get no pages are an ordinary outcome: plan, write, trees, move and trim leave no error, rows without
    a place read as zeros, and the others' results are what they are."""
    s = _Step(va, kind, old, new, width, page, heads, kv, 64, free=free)
    _ok(va)
    lost, table = s.plan.unplaced.tolist(), s.table.tolist()
    assert max(lost) > 0 and min(lost) == 0 or free == 0
    for b, n in enumerate(new):
        assert lost[b] == sum(s.place(b, old[b] + i) < 0 for i in range(n))
        assert (-1 in table[b]) == (lost[b] > 0)
    s.attend()
    _ok(va)
    s.attend(20)
    _ok(va)
    s.keep([sorted({0, n // 3, n - 1} if b % 2 or lost[b] else {0, min(2, n - 1)}) for b, n in enumerate(new)])
    _ok(va)


def test_the_same_step_undone(va):
    """Nothing kept: lengths, stack and count are as before the step."""
    old, new, width, page, free = SHORT[0]
    s = _Step(va, "bf16", old, new, width, page, 1, 1, 64, free=free)
    s.keep([[]] * len(old))
    _ok(va)
    assert s.seqlens.tolist() == old and s.pool.free_count.item() == free and s.pool.free_pages[:free].tolist() == s.stack


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [1, 32])
@pytest.mark.parametrize("bad", [-2, -2147483648, 1 << 20])
def test_other_entries_are_reported(va, kind, heads, bad):
    """An entry that is no page and not the plan's -1 is an error in the trees and in move, as it was; the causal band and the
    packed write, which have no plan, report -1 too."""
    cache, _, _ = C.make_cache([60], 1, 64, 16, kind, DEV)
    q = torch.randn(4, heads, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    masks, cu = torch.full((4, 1), -1, dtype=torch.int32, device=DEV), C.cu_of([4], DEV)
    for entry, want in ((-1, 0), (bad, va.VARLEN_ERR_DEVICE_BOUNDS)):
        cache.block_table[0, 3] = entry
        va.attention_fwd_paged_tree(q, cache, cu, masks, max_seqlen_q=4)
        _ok(va, want)
        va.cache_move(cache, cu, _ints([[0, 2]]), _ints([2]))
        _ok(va, want)
    cache.block_table[0, 3] = -1
    va.attention_fwd_paged(q, cache, cu, max_seqlen_q=4, causal=True)
    _ok(va, va.VARLEN_ERR_DEVICE_BOUNDS)
    va.cache_write(cache, q[:, :1], q[:, :1], cu)
    _ok(va, va.VARLEN_ERR_DEVICE_BOUNDS)


def test_moves_past_the_table_are_passed_over(va):
    """Rows that the plan could not place past the table's end go nowhere and come from nowhere, without an error."""
    s = _Step(va, "bf16", [70, 0], [40, 6], 5, 16, 2, 2, 64)
    s.keep([[0, 4, 9, 10, 30, 39], [1, 3, 5]])
    _ok(va)
