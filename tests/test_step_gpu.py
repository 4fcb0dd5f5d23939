"""A step's lists (plan, trim, move), rotary positions and the cache write behind them, on a GPU: against loops over
whole numbers, 64-bit forms and the calls that they stand for."""
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


def _ok(va, want=0):
    st = va.varlen_attn_get_device_status()
    assert st == want, va.varlen_attn_status_string(st)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _rows(n, heads, dim, seed, pad=0, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.full((n, heads, dim + pad), math.nan, dtype=torch.bfloat16)
    x[..., :dim] = (torch.randn(n, heads, dim, generator=g) * amp).to(torch.bfloat16)
    return x.to(DEV)[..., :dim]


# ------------------------------------------------------------------ rotary positions

def _check_turned(got, x, angle, rot, inter, scale, back=False):
    """The angle is held to 2^-32 turn and rounded to fp32 twice (below 0.79: 3 2^-24 in all), sine and cosine add
    2 2^-24, the scale 2^-24, the two products and their sum 2 2^-24: 8 2^-24 of scale (|x1| + |x2|); then one
    rounding to bf16."""
    y, size = S.turned(x, angle.to(x.device), rot, inter, scale, back)
    d = (got.double() - y).abs()
    tol = 8 * 2.0 ** -24 * size + 2.0 ** -8 * y.abs() + 1e-38
    assert (d <= tol).all(), "off by %.3g, worst ratio %.3g" % (d.max(), (d / tol).max())
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 8), (64, 40), (96, 96), (96, 24), (96, 48), (128, 128), (128, 32), (128, 72), (128, 16)])
@pytest.mark.parametrize("inter", [False, True])
def test_rotary(va, dim, rot, inter):
    total, H, Hk = 67, 5, 3
    freq, scale = va.rotary_frequencies(rot, 500000.0, stretch=4.0)
    rope = va.Rotary(freq, interleaved=inter, scale=scale, device=DEV)
    pos = torch.randint(-(1 << 20), 1 << 22, (total,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    pos[:4] = torch.tensor([0, 1, -1, (1 << 24) + 3], dtype=torch.int32)
    q, k = _rows(total, H, dim, 2, pad=32), _rows(total, Hk, dim, 3, amp=100.0)
    angle = pos.double()[:, None] * freq
    scale = float(torch.tensor(scale, dtype=torch.float32))
    for back, call in ((False, va.rotary), (True, va.rotary_bwd)):
        qo, ko = call(q, k, rope, positions=pos.to(DEV))
        _ok(va)
        _check_turned(qo, q, angle, rot, inter, scale, back)
        _check_turned(ko, k, angle, rot, inter, scale, back)
        # in place, the same bits, nothing between the rows
        q2 = _rows(total, H, dim, 2, pad=32)
        out, none = call(q2, None, rope, pos.to(DEV), None, q2)
        assert none is None and out is q2 and torch.equal(q2, qo)
        whole = q2.as_strided((total, H, dim + 32), (H * (dim + 32), dim + 32, 1))
        assert torch.isnan(whole[..., dim:]).all()
        _ok(va)


def test_rotary_far_positions(va):
    """Any int32 position: the angle is a whole-number product."""
    pos = [0, 1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -7, 185619, 2 ** 24 + 1]
    st, turns = va.varlen_attn_rotary_turns([1.0, 0.25, 1e-3, 2 * math.pi - 1e-9, 0.0, -0.5, 3.0, 100.0])
    assert st == 0
    rope = va.Rotary([1.0, 0.25, 1e-3, 2 * math.pi - 1e-9, 0.0, -0.5, 3.0, 100.0], device=DEV)
    q = _rows(len(pos), 2, 64, 5)
    out, _ = va.rotary(q, None, rope, positions=_ints(pos))
    _ok(va)
    _check_turned(out, q, S.angles(pos, turns), 16, False, 1.0)


@pytest.mark.parametrize("lens,pad", [([1], 0), ([0, 37, 0, 100], 3), ([5, 0, 0], 0), ([3] * 70 + [0] * 40 + [200], 9), ([4000], 0)])
def test_rotary_in_segments(va, lens, pad):
    """Rows stand at their places in their segments; rows outside every segment are not written."""
    total, H, Hk, dim = sum(lens) + pad, 7, 1, 96
    freq, _ = va.rotary_frequencies(dim)
    rope = va.Rotary(freq, device=DEV)
    q, k = _rows(total, H, dim, 2), _rows(total, Hk, dim, 3)
    qo = torch.full_like(q, 7.0)
    ko = torch.full((total, 2, dim), 7.0, dtype=torch.bfloat16, device=DEV)[:, 1:]
    va.rotary(q, k, rope, cu_seqlens=C.cu_of(lens, DEV), q_out=qo, k_out=ko)
    _ok(va)
    at = torch.cat([torch.arange(n) for n in lens])
    n = sum(lens)
    _check_turned(qo[:n], q[:n], at.double()[:, None] * freq, dim, False, 1.0)
    _check_turned(ko[:n], k[:n], at.double()[:, None] * freq, dim, False, 1.0)
    assert (qo[n:] == 7.0).all() and (ko[n:] == 7.0).all()


def test_rotary_gradient_is_the_transpose(va):
    """<turn(x), g> = <x, turn_bwd(g)>, and differences: both maps are linear, so a unit step of one element shows the
    column of one and the row of the other.  Elements of sizes that bf16 holds exactly leave only the outputs' own
    roundings."""
    dim, rot = 64, 32
    freq, _ = va.rotary_frequencies(rot)
    rope = va.Rotary(freq, interleaved=True, scale=1.5, device=DEV)
    pos = _ints([12345] * dim)
    eye = torch.eye(dim, device=DEV, dtype=torch.bfloat16)[:, None]  # row r: the step of element r
    cols, _ = va.rotary(eye, None, rope, positions=pos)
    rows, _ = va.rotary_bwd(eye, None, rope, positions=pos)
    _ok(va)
    assert torch.equal(cols[:, 0], rows[:, 0].T)
    zero, _ = va.rotary(torch.zeros_like(eye), None, rope, positions=pos)
    assert (zero == 0).all()


def test_rotary_broadcast_input_and_long_strides(va):
    """One head read as many (zero head stride), and rows more than 2^31 elements apart."""
    freq, _ = va.rotary_frequencies(128)
    rope = va.Rotary(freq, device=DEV)
    one = _rows(9, 1, 128, 4)
    qo, _ = va.rotary(one.expand(-1, 6, -1), None, rope, positions=_ints(list(range(9))))
    ref, _ = va.rotary(one.repeat(1, 6, 1), None, rope, positions=_ints(list(range(9))))
    assert torch.equal(qo, ref)
    base = torch.zeros((1 << 31) + 4096, dtype=torch.bfloat16, device=DEV)
    far = base.as_strided((3, 6, 128), (1 << 30, 128, 1))
    far.copy_(one[:3].expand(-1, 6, -1))
    va.rotary(far, None, rope, _ints([0, 1, 2]), None, far)
    _ok(va)
    assert torch.equal(far, ref[:3])


# ------------------------------------------------------------------ the cache write behind it

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,rot,inter", [(64, 64, False), (64, 24, True), (96, 96, False), (96, 8, False), (128, 128, True), (128, 64, False), (128, 120, True)])
@pytest.mark.parametrize("page,order,heads", [(16, "nhd", 1), (64, "hnd", 3), (32, "together", 9)])
def test_rotary_cache_write(va, kind, dim, rot, inter, page, order, heads):
    """The bits of rotary followed by cache_write, whole pools."""
    lens, new, H = [40, 1, 130, 17], [7, 1, 130, 0], 6
    total, extra = sum(new), 4
    freq, _ = va.rotary_frequencies(rot)
    rope = va.Rotary(freq, interleaved=inter, device=DEV)
    q, k, v = _rows(total + extra, H, dim, 1), _rows(total + extra, heads, dim, 2, pad=16), _rows(total + extra, heads, dim, 3)
    if kind == "e4m3":  # vectors of zeros, infinities and NaN keep their own rules
        k[0], k[1, 0, 3], v[2, 0, 5], v[3] = 0, math.inf, math.nan, 0
    pos, slots = [], []
    a, _, _ = C.make_cache(lens, heads, dim, page, kind, DEV, seed=3, order=order)
    b, _, _ = C.make_cache(lens, heads, dim, page, kind, DEV, seed=3, order=order)
    table = a.block_table.tolist()
    for s, n in enumerate(new):
        for i in range(lens[s] - n, lens[s]):
            pos.append(i)
            slots.append(table[s][i // page] * page + i % page)
    pos, slots = _ints(pos + [5] * extra), _ints(slots + [-1] * extra, torch.int64)
    q1 = va.rotary_cache_write(a, q, k, v, rope, pos, slots)
    q2, k2 = va.rotary(q, k, rope, positions=pos)
    va.cache_write(b, k2, v, C.cu_of(new, DEV))
    _ok(va)
    assert torch.equal(q1.view(torch.int16), q2.view(torch.int16))
    for x, y in ((a.k_pages, b.k_pages), (a.v_pages, b.v_pages)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
    if kind == "e4m3":
        for x, y in ((a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    # no queries; queries in place
    assert va.rotary_cache_write(a, None, k, v, rope, pos, slots) is None
    assert va.rotary_cache_write(a, q, k, v, rope, pos, slots, q_out=q) is q and torch.equal(q.view(torch.int16), q2.view(torch.int16))
    _ok(va)


def test_rotary_cache_write_slots(va):
    """Slots past the last page are passed over and recorded, negative ones only passed over."""
    cache, _, _ = C.make_cache([16], 2, 64, 16, "bf16", DEV)
    before = cache.k_pages.clone()
    rope = va.Rotary(va.rotary_frequencies(64)[0], device=DEV)
    x = _rows(3, 2, 64, 1)
    last = cache.k_pages.shape[0] * 16
    va.rotary_cache_write(cache, None, x, x, rope, _ints([0, 1, 2]), _ints([-1, -5, -(1 << 62)], torch.int64))
    _ok(va)
    assert torch.equal(cache.k_pages.view(torch.int16), before.view(torch.int16))
    va.rotary_cache_write(cache, None, x, x, rope, _ints([0, 1, 2]), _ints([last, 1 << 40, last - 1], torch.int64))
    _ok(va, va.VARLEN_ERR_DEVICE_BOUNDS)
    assert torch.equal(cache.v_pages[-1, -1], x[2])
    before[-1, -1] = cache.k_pages[-1, -1]
    assert torch.equal(cache.k_pages.view(torch.int16), before.view(torch.int16))


# ------------------------------------------------------------------ plan and trim

def _pool(va, old, width, page, free, count, seed=0, apart=False):
    """A pool whose sequences own random pages; returns (pool, table as lists)."""
    need = [-(-min(n, width * page) // page) for n in old]
    g = torch.Generator().manual_seed(seed)
    names = torch.randperm(sum(need) + free, generator=g).tolist()
    table, at = [], 0
    for n in need:
        table.append(names[at:at + n] + [-9] * (width - n))
        at += n
    stack = names[at:] + [-9] * at
    t = torch.full((len(old), width + 3), -9, dtype=torch.int32, device=DEV)[:, :width]
    t.copy_(_ints(table).reshape(len(old), width))
    more = (_ints([-1] * len(old)), _ints([-1])) if apart else (None, None)
    return va.PagePool(t, _ints(old), _ints(stack), _ints([count]), page, *more), table, stack


def _check_plan(va, old, new, total, page, width, free, count=None, trees=False, words=0, seed=0, apart=False, status=0, parents=None):
    count = free if count is None else count
    pool, table, stack = _pool(va, old, width, page, free, count, seed, apart)
    step = va.StepPlan(len(old), total, DEV, mask_words=words)
    for t, x in ((step.slots, 77), (step.positions, 77), (step.unplaced, 77), (step.cu_seqlens, 77)):
        t.fill_(x)
    if trees and parents is None:
        g = torch.Generator().manual_seed(seed + 1)
        parents, left = [], total
        for n in new:
            n = min(max(n, 0), left)
            parents += S.random_tree(n, g)
            left -= n
        parents += [3] * left
    if trees:
        step.masks.fill_(77)
    ref = S.plan(new, total, old, table, stack, count, page, parents if trees else None, words)
    got = va.cache_plan(pool, step, _ints(new), parents=_ints(parents) if trees else None)
    assert got is step
    _ok(va, status)
    assert step.cu_seqlens.tolist() == ref["cu"]
    assert pool.seqlens_out.tolist() == ref["seqlens"]
    assert pool.free_count_out.tolist() == [ref["count"]]
    assert pool.block_table.tolist() == ref["table"]
    assert step.slots.tolist() == ref["slots"]
    assert step.positions.tolist() == ref["positions"]
    assert step.unplaced.tolist() == ref["unplaced"]
    assert pool.free_pages.tolist() == stack
    if trees:
        assert torch.equal(step.masks.cpu(), ref["masks"])
    if apart:
        assert pool.seqlens.tolist() == old and pool.free_count.tolist() == [count]
    return pool, step, ref, stack


PLANS = [
    # old lengths, new rows, rows of the buffers beyond them, page, table width, free pages
    ([0], [1], 0, 16, 1, 1),
    ([0, 15, 16, 17, 31], [1, 1, 1, 1, 1], 3, 16, 4, 9),
    ([100, 0, 7], [0, 0, 0], 5, 32, 8, 4),
    ([5, 0, 64, 100, 3], [0, 200, 1, 28, 61], 0, 64, 8, 20),
    ([8191] * 300, [1] * 300, 20, 16, 513, 400),
    ([n % 40 for n in range(1024)], [n % 3 for n in range(1024)], 1, 16, 4, 2000),
    ([n % 40 for n in range(1500)], [n % 3 for n in range(1500)], 7, 16, 4, 3000),
    ([0, 0, 0], [5000, 0, 1234], 100, 128, 64, 60),
    ([3], [70000], 0, 1024, 70, 70),
]


@pytest.mark.parametrize("case", PLANS)
@pytest.mark.parametrize("apart", [False, True])
def test_plan(va, case, apart):
    old, new, extra, page, width, free = case
    _check_plan(va, old, new, sum(new) + extra, page, width, free, apart=apart)


@pytest.mark.parametrize("case", [c for c in PLANS if max(c[1]) <= 4096])
def test_plan_trees(va, case):
    old, new, extra, page, width, free = case
    words = -(-max(max(new), 1) // 32)
    _check_plan(va, old, new, sum(new) + extra, page, width, free, trees=True, words=words)
    _check_plan(va, old, new, sum(new) + extra, page, width, free, trees=True, words=min(words + 3, 128), seed=5)


@pytest.mark.parametrize("n,words,shape", [(4096, 128, "chain"), (4096, 128, "comb"), (4000, 127, "star"), (2048, 64, "comb"),
                                           (33, 2, "chain"), (31, 4, "comb"), (1000, 32, "mixed")])
def test_plan_deep_trees(va, n, words, shape):
    parents = {"chain": [i - 1 for i in range(n)], "comb": [-1, 0] + [i - 2 + (i % 2 == 0) * 0 for i in range(2, n)],
               "star": [-1] + [0] * (n - 1), "mixed": S.random_tree(n, torch.Generator().manual_seed(3), chain=0.9)}[shape]
    _check_plan(va, [20, 0], [n, 3], n + 3, 16, 300, 300, trees=True, words=words, parents=parents + [-1, 0, 0])


def test_plan_without_enough_pages(va):
    """The running need decides, first come first served; who gets nothing keeps what it has, with -1 behind."""
    old, new = [10, 0, 14, 30, 16], [7, 40, 1, 2, 1]  # need 1, 3, 0, 0, 1
    for free in range(7):
        _check_plan(va, old, new, sum(new) + 2, 16, 5, 6, count=min(free, 6))
        _check_plan(va, old, new, sum(new) + 2, 16, 5, 6, count=min(free, 6), trees=True, words=2)
    _check_plan(va, [10, 79, 70], [7, 2, 11], 20, 16, 5, 6)  # past the table's width: none
    _check_plan(va, [10, 200, 70], [7, 2, 10], 19, 16, 5, 6)
    _check_plan(va, [n % 40 for n in range(1500)], [n % 3 for n in range(1500)], 1600, 16, 4, 300)


def test_plan_clamps(va):
    """Negative lengths count as none, rows past the buffers do not exist, counts stay in their range."""
    _check_plan(va, [5, -3, 0], [-4, 10, 6], 12, 16, 4, 8)
    _check_plan(va, [5, 3, 0], [2 ** 31 - 1, 10, 2 ** 31 - 1], 40, 16, 4, 8)
    _check_plan(va, [5, 3, 0], [4, 4, 4], 0, 16, 4, 8)
    # a count past the stack's end counts as all of it: its last entry, which names no page here, is found out
    pool, table, stack = _pool(va, [5], 4, 16, 8, 1000)
    step = va.StepPlan(1, 30, DEV)
    va.cache_plan(pool, step, _ints([20]))
    _ok(va, va.VARLEN_ERR_DEVICE_BOUNDS)
    assert pool.free_count.tolist() == [len(stack) - 1] and stack[-1] == -9
    assert step.slots.tolist() == [table[0][0] * 16 + i for i in range(5, 16)] + [-1] * 19
    # where every entry names a page, all is well
    pool, table, stack = _pool(va, [0], 4, 16, 8, 1000)
    va.cache_plan(pool, step, _ints([20]))
    _ok(va)
    assert pool.free_count.tolist() == [len(stack) - 2] and pool.block_table[0, :2].tolist() == stack[:-3:-1]


def test_plan_bad_trees(va):
    """Parents that are not before their row count as none; rows that no mask can name have none; both are recorded."""
    _check_plan(va, [5], [6], 8, 16, 4, 8, trees=True, words=1, parents=[-1, 1, 0, 77, 3, -100, 0, 0], status=va.VARLEN_ERR_DEVICE_BOUNDS)
    g = torch.Generator().manual_seed(2)
    _check_plan(va, [5, 0], [40, 4], 44, 16, 4, 8, trees=True, words=1, parents=S.random_tree(32, g) + [31] * 8 + [-1, 0, 1, 2],
                status=va.VARLEN_ERR_DEVICE_BOUNDS)
    g = torch.Generator().manual_seed(2)
    _check_plan(va, [5, 0], [3000, 4], 3004, 16, 200, 200, trees=True, words=3, parents=S.random_tree(96, g) + [31] * 2904 + [-1, 0, 1, 2],
                status=va.VARLEN_ERR_DEVICE_BOUNDS)


@pytest.mark.parametrize("case", PLANS)
def test_trim_undoes_a_plan(va, case):
    """Back to the old lengths, both ways of saying so: the stack is what it was, order included."""
    old, new, extra, page, width, free = case
    for by_step in (False, True):
        pool, step, ref, stack = _check_plan(va, old, new, sum(new) + extra, page, width, free)
        va.cache_trim(pool, _ints([0] * len(old)) if by_step else _ints(old), step.cu_seqlens if by_step else None)
        _ok(va)
        assert pool.seqlens.tolist() == old and pool.free_count.tolist() == [free] and pool.free_pages.tolist() == stack


@pytest.mark.parametrize("batch,width,page", [(1, 1, 16), (5, 7, 16), (70, 40, 32), (1500, 6, 16), (2, 5000, 16)])
def test_trim(va, batch, width, page):
    g = torch.Generator().manual_seed(batch)
    old = torch.randint(0, width * page + 1, (batch,), generator=g).tolist()
    keep = [int(n * u) if u < 0.8 else n + 5 for n, u in zip(old, torch.rand(batch, generator=g).tolist())]
    keep[0] = -3
    pool, table, stack = _pool(va, old, width, page, 4, 2, apart=True)
    holes = []  # entries that a step without pages left
    for b in range(0, batch, 3):
        if old[b] > page:
            pool.block_table[b, (old[b] - 1) // page] = -1
            holes.append((b, (old[b] - 1) // page))
    va.cache_trim(pool, _ints(keep))
    _ok(va)
    want = [min(max(k, 0), n) for k, n in zip(keep, old)]
    assert pool.seqlens_out.tolist() == want and pool.seqlens.tolist() == old
    back = [table[b][i] for b in reversed(range(batch)) for i in reversed(range(-(-want[b] // page), -(-old[b] // page))) if (b, i) not in holes]
    assert pool.free_count_out.tolist() == [2 + len(back)]
    assert pool.free_pages.tolist()[:2 + len(back)] == stack[:2] + back


def test_trim_records_what_it_cannot_put_back(va):
    pool, table, stack = _pool(va, [40, 40], 4, 16, 2, 2)
    pool.block_table[0, 1] = 1000
    va.cache_trim(pool, _ints([0, 40]))
    _ok(va, va.VARLEN_ERR_DEVICE_BOUNDS)
    assert pool.free_pages.tolist()[:4] == stack[:2] + [table[0][2], table[0][0]] and pool.free_count.tolist() == [4]
    pool, table, stack = _pool(va, [40, 40], 4, 16, 2, 2)
    full = torch.full((8,), 5, dtype=torch.int32, device=DEV)
    tight = va.PagePool(pool.block_table, pool.seqlens, full[:7], _ints([6]), 16)
    va.cache_trim(tight, _ints([0, 40]))
    _ok(va, va.VARLEN_ERR_DEVICE_BOUNDS)
    first = [i for i in reversed(table[0][:3]) if i < 7][0]  # (a pool of 7 has no page 7)
    assert tight.free_count.tolist() == [7] and full.tolist() == [5] * 6 + [first, 5]


# ------------------------------------------------------------------ accepted rows

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,page,order,heads,layers", [(64, 16, "nhd", 1, 1), (96, 32, "hnd", 3, 2), (128, 16, "together", 8, 1), (128, 64, "padded", 17, 3)])
def test_move(va, kind, dim, page, order, heads, layers):
    lens, new = [40, 0, 100, 17, 200, 9], [30, 0, 70, 17, 5, 12]  # the last holds fewer positions than rows came
    kept = [[0, 3, 4, 20, 29], [], list(range(1, 70)), [16], [2, 4], [1, 5, 11]]
    most = max(len(k) for k in kept)
    caches = [C.make_cache(lens, heads, dim, page, kind, DEV, seed=3, order=order)[0] for _ in range(layers)]
    caches = [caches[0]] + [va.PagedCache(c.k_pages, c.v_pages, caches[0].block_table, caches[0].seqlens, c.k_scale, c.v_scale)
                            for c in caches[1:]]
    for i, c in enumerate(caches):  # layers differ
        c.k_pages.view(torch.uint8)[..., 0] = i
    tables = caches[0].block_table.tolist()
    want = []
    for c in caches:
        pools = [c.k_pages.contiguous().view(torch.uint8), c.v_pages.contiguous().view(torch.uint8)]
        pools = [p.clone() for p in pools] + [s.clone() for s in (c.k_scale, c.v_scale) if s is not None]
        old = [p.clone() for p in pools]
        for b, rows in enumerate(kept):
            for i, r in enumerate(rows):
                src, dst = lens[b] - new[b] + r, lens[b] - new[b] + i
                if dst < 0 or src < 0:
                    continue
                sp, dp = tables[b][src // page], tables[b][dst // page]
                for n, p in enumerate(pools):
                    if n < 2:
                        p[dp, dst % page] = old[n][sp, src % page]
                    else:
                        p[dp, :, dst % page] = old[n][sp, :, src % page]
        want.append(pools)
    k = torch.full((len(lens), most + 2), 999, dtype=torch.int32, device=DEV)
    for b, rows in enumerate(kept):
        k[b, :len(rows)] = _ints(rows)
    va.cache_move(caches if layers > 1 else caches[0], C.cu_of(new, DEV), k[:, :most], _ints([len(r) for r in kept]))
    _ok(va)
    for c, pools in zip(caches, want):
        got = [c.k_pages.contiguous().view(torch.uint8), c.v_pages.contiguous().view(torch.uint8)]
        got += [s for s in (c.k_scale, c.v_scale) if s is not None]
        for x, y in zip(got, pools):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_move_many_layers_and_bad_rows(va):
    """More caches than one launch takes; rows outside [i, n) move nothing and are recorded."""
    first, _, _ = C.make_cache([50], 1, 64, 16, "bf16", DEV, seed=1)
    pools = [torch.randn_like(first.k_pages) for _ in range(140)]
    caches = [va.PagedCache(pools[2 * i], pools[2 * i + 1], first.block_table, first.seqlens) for i in range(70)]
    before = [p.clone() for p in pools]
    va.cache_move(caches, C.cu_of([20], DEV), _ints([[3, 7]]), _ints([2]))
    _ok(va)
    row = first.block_table[0].long()
    for p, o in zip(pools, before):
        o[row[30 // 16], 30 % 16], o[row[31 // 16], 31 % 16] = o[row[33 // 16], 33 % 16].clone(), o[row[37 // 16], 37 % 16].clone()
        assert torch.equal(p, o)
    va.cache_move(caches[0], C.cu_of([20], DEV), _ints([[0, 0, 20, -1, 9]]), _ints([9]))
    _ok(va, va.VARLEN_ERR_DEVICE_BOUNDS)
    before[0][row[34 // 16], 34 % 16] = before[0][row[39 // 16], 39 % 16].clone()
    assert torch.equal(pools[0], before[0])


def test_far_pages(va):
    """Pages past 2^32 bytes: written, moved and read back."""
    pages, page, heads, dim = 150000, 16, 8, 128
    k = torch.zeros(pages, page, heads, dim, dtype=torch.bfloat16, device=DEV)
    table = _ints([[pages - 1, pages - 2, 149000]])
    cache = va.PagedCache(k, k.clone(), table, _ints([40]))
    rope = va.Rotary([0.0] * 64, device=DEV)  # a turn by nothing
    x, y = _rows(40, heads, dim, 1), _rows(40, heads, dim, 2)
    pos = torch.arange(40, dtype=torch.int32, device=DEV)
    slots = table[0].long()[pos.long() // page] * page + pos.long() % page
    va.rotary_cache_write(cache, None, x, y, rope, pos, slots)
    va.cache_move(cache, C.cu_of([30], DEV), _ints([[5, 29]]), _ints([2]))
    _ok(va)
    x[10], x[11], y[10], y[11] = x[15].clone(), x[39].clone(), y[15].clone(), y[39].clone()
    ko, vo = va.cache_read(cache, C.cu_of([40], DEV), 40)
    assert torch.equal(ko, x) and torch.equal(vo, y)
