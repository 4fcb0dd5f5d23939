"""Refusals of a step's entry points (plan, trim, move, rotary positions, the cache write behind them, tree attention),
on the CPU: status codes for arguments they must not accept (fake pointers, never followed: every call fails validation
or stops at the device query), the binding's own checks, and what is computed on the host."""
import ctypes
import math

import pytest
import torch

from tests.test_paged_abi import _cache, _tensors, va  # noqa: F401  (va: the fixture)


def _runs(va):
    return (va.VARLEN_ERR_CUDA, va.VARLEN_ERR_ARCH)


def _pool(va, **kw):
    c = va.VarlenPagePool()
    c.block_table, c.seqlens, c.seqlens_out, c.free_pages, c.free_count, c.free_count_out = (
        0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000)
    c.table_stride, c.num_pages, c.page_size, c.max_pages = 8, 10, 16, 8
    for n, x in kw.items():
        setattr(c, n, x)
    return c


def _plan(va, pool, new=0x100, batch=3, parents=None, total=10, cu=0x200, slots=0x300, pos=0x400, un=0x500, masks=None,
          words=0, ws=0x10000, nb=1 << 30):
    return va.LIB.varlen_attn_cache_plan(ctypes.byref(pool) if pool else None, new, batch, parents, total, cu, slots, pos,
                                         un, masks, words, ws, nb, None)


def _trim(va, pool, lens=0x100, cu=None, batch=3):
    return va.LIB.varlen_attn_cache_trim(ctypes.byref(pool) if pool else None, lens, cu, batch, None)


POOL = [({"num_pages": 0}, "SHAPE"), ({"num_pages": -1}, "SHAPE"), ({"page_size": 8}, "SHAPE"), ({"page_size": 48}, "SHAPE"),
        ({"page_size": 2048}, "SHAPE"), ({"max_pages": -1}, "SHAPE"), ({"max_pages": 1 << 27, "table_stride": 1 << 27}, "SHAPE"),
        ({"table_stride": 7}, "STRIDE"), ({"table_stride": -1}, "STRIDE"), ({"block_table": None}, "NULL"), ({"seqlens": None}, "NULL"),
        ({"seqlens_out": None}, "NULL"), ({"free_pages": None}, "NULL"), ({"free_count": None}, "NULL"), ({"free_count_out": None}, "NULL")]


@pytest.mark.parametrize("change,code", POOL)
def test_pool_refusals(va, change, code):
    code = getattr(va, "VARLEN_ERR_" + code)
    assert _plan(va, _pool(va, **change)) == code
    assert _trim(va, _pool(va, **change)) == code


def test_pool_edges(va):
    for kw in ({}, {"max_pages": 0, "block_table": None, "table_stride": 0}, {"page_size": 1024}, {"table_stride": 1 << 30}):
        assert _plan(va, _pool(va, **kw)) in _runs(va), kw
        assert _trim(va, _pool(va, **kw)) in _runs(va), kw
    assert _plan(va, _pool(va, table_stride=0), batch=1) in _runs(va)  # a stride over one row is not used
    assert _plan(va, None) == _trim(va, None) == va.VARLEN_ERR_NULL


def test_plan_refusals(va):
    p = _pool(va)
    for batch in (0, -1, (1 << 20) + 1):
        assert _plan(va, p, batch=batch) == _trim(va, p, batch=batch) == va.VARLEN_ERR_SHAPE
    assert _plan(va, _pool(va, max_pages=1 << 12, table_stride=1 << 12), batch=1 << 20) == va.VARLEN_ERR_SHAPE  # 2^32 entries
    for total in (-1, 2 ** 31 - 1):
        assert _plan(va, p, total=total) == va.VARLEN_ERR_SHAPE
    for name in ("new", "cu", "slots", "pos", "un"):
        assert _plan(va, p, **{name: None}) == va.VARLEN_ERR_NULL
    assert _plan(va, p, slots=None, pos=None, total=0) in _runs(va)
    assert _plan(va, p, slots=0x304) == va.VARLEN_ERR_ALIGN
    for words in (0, -1, 129):
        assert _plan(va, p, parents=0x700, masks=0x800, words=words) == va.VARLEN_ERR_SHAPE
    assert _plan(va, p, parents=0x700, words=4) == va.VARLEN_ERR_NULL
    assert _plan(va, p, parents=0x700, masks=0x800, words=128) in _runs(va)
    need = va.varlen_attn_cache_plan_workspace_size(3)
    for ws, nb in ((None, need), (0x10008, need), (0x10000, need - 1)):
        assert _plan(va, p, ws=ws, nb=nb) == va.VARLEN_ERR_WORKSPACE
    assert _plan(va, p, nb=need) in _runs(va)
    assert va.varlen_attn_cache_plan_workspace_size(-1) == va.varlen_attn_cache_plan_workspace_size((1 << 20) + 1) == 0
    assert _trim(va, p, lens=None) == va.VARLEN_ERR_NULL


def _move(va, caches, count=None, cu=0x100, batch=1, total=10, kept=0x200, stride=4, lens=0x300, most=4):
    arr = (va.VarlenKvCache * len(caches))(*caches) if caches else None
    return va.LIB.varlen_attn_cache_move(arr, len(caches) if count is None else count, cu, batch, total, kept, stride, lens, most,
                                         None)


def test_move_refusals(va):
    c = _cache(va)
    assert _move(va, [c]) in _runs(va) and _move(va, [c, c, c]) in _runs(va)
    for kind in (0, 1):
        assert _move(va, [_cache(va, type=kind)]) in _runs(va)
    assert _move(va, None, count=1) == va.VARLEN_ERR_NULL
    for count in (0, -1, 1025):
        assert _move(va, [c], count=count) == va.VARLEN_ERR_SHAPE
    assert _move(va, [c], total=-1) == _move(va, [c], most=-1) == _move(va, [c], batch=0) == va.VARLEN_ERR_SHAPE
    assert _move(va, [c], cu=None) == _move(va, [c], lens=None) == _move(va, [c], kept=None) == va.VARLEN_ERR_NULL
    assert _move(va, [c], stride=-1) == va.VARLEN_ERR_STRIDE
    assert _move(va, [c], kept=None, most=0) in _runs(va)
    # layers that are not alike, or not over one table
    for change in ({"type": 1}, {"num_pages": 11}, {"page_size": 32}, {"max_pages": 7}, {"num_kv_heads": 1}, {"head_dim": 96},
                   {"block_table": 0x30010}, {"seqlens": 0x40010}, {"table_stride": 9}, {"sk": va.VarlenPageStride(4096, 128, 64)}):
        kw = dict(change)
        if kw.get("type") == 1:
            d = _cache(va, type=1)
        else:
            d = _cache(va)
            for n, x in kw.items():
                setattr(d, n, x)
            if "page_size" in kw or "head_dim" in kw:
                d = _cache(va, **kw)
        assert _move(va, [c, d]) == va.VARLEN_ERR_SHAPE, change
    d = _cache(va)
    d.k = None
    assert _move(va, [c, d]) == va.VARLEN_ERR_NULL


def _rope(va, **kw):
    r = va.VarlenRotary()
    r.turns, r.rotary_dim, r.interleaved, r.scale = 0x9000, 64, 0, 1.0
    for n, x in kw.items():
        setattr(r, n, x)
    return r


ROPE = [({"rotary_dim": 0}, "SHAPE"), ({"rotary_dim": 12}, "SHAPE"), ({"rotary_dim": 72}, "SHAPE"), ({"rotary_dim": -8}, "SHAPE"),
        ({"interleaved": 2}, "SHAPE"), ({"interleaved": -1}, "SHAPE"), ({"scale": math.inf}, "SHAPE"), ({"scale": math.nan}, "SHAPE"),
        ({"turns": None}, "NULL"), ({"turns": 0x9004}, "ALIGN")]


def _rotary(va, rope=None, q=0x1000, sq=(256, 64), k=0x2000, sk=(128, 64), pos=0x100, cu=None, batch=0, total=10, heads=4, kv=2,
            dim=64, qo=0x3000, sqo=(256, 64), ko=0x4000, sko=(128, 64), inverse=0):
    S = va.VarlenStride
    rope = _rope(va) if rope is None else rope
    return va.LIB.varlen_attn_rotary(q, S(*sq), k, S(*sk), pos, cu, batch, total, heads, kv, dim, ctypes.byref(rope) if rope else None,
                                     inverse, qo, S(*sqo), ko, S(*sko), None)


def _write(va, c=None, rope=None, q=0x1000, sq=(256, 64), k=0x2000, v=0x2800, st=(128, 64), pos=0x100, slots=0x200, total=10, heads=4,
           qo=0x3000, sqo=(256, 64)):
    S = va.VarlenStride
    c, rope = _cache(va) if c is None else c, _rope(va) if rope is None else rope
    return va.LIB.varlen_attn_rotary_cache_write(q, S(*sq), k, S(*st), v, S(*st), pos, slots, total, heads,
                                                 ctypes.byref(c) if c else None, ctypes.byref(rope) if rope else None, qo, S(*sqo), None)


@pytest.mark.parametrize("change,code", ROPE)
def test_rotary_struct_refusals(va, change, code):
    code = getattr(va, "VARLEN_ERR_" + code)
    assert _rotary(va, _rope(va, **change)) == code
    assert _write(va, rope=_rope(va, **change)) == code


def test_rotary_refusals(va):
    assert _rotary(va) in _runs(va) and _rotary(va, inverse=1) in _runs(va)
    assert _rotary(va, rope=0) == va.VARLEN_ERR_NULL
    assert _rotary(va, k=None, ko=None, kv=0) in _runs(va) and _rotary(va, q=None, qo=None, heads=0) in _runs(va)
    assert _rotary(va, heads=0, kv=0) == _rotary(va, heads=-1) == _rotary(va, kv=-1) == _rotary(va, total=-1) == va.VARLEN_ERR_SHAPE
    assert _rotary(va, heads=1 << 20) == va.VARLEN_ERR_SHAPE
    for dim in (32, 80, 256):
        assert _rotary(va, dim=dim) == va.VARLEN_ERR_HEAD_DIM
    assert _rotary(va, pos=None) == va.VARLEN_ERR_NULL
    assert _rotary(va, pos=None, cu=0x500, batch=1) in _runs(va)
    assert _rotary(va, pos=None, cu=0x500, batch=0) == _rotary(va, pos=None, cu=0x500, batch=(1 << 30) + 1) == va.VARLEN_ERR_SHAPE
    for name in ("q", "k", "qo", "ko"):
        assert _rotary(va, **{name: None}) == va.VARLEN_ERR_NULL
        assert _rotary(va, **{name: 0x1008}) == va.VARLEN_ERR_ALIGN
    for stride in ((-8, 64), (256, 60), (1 << 39, 64)):
        for name in ("sq", "sk", "sqo", "sko"):
            assert _rotary(va, **{name: stride}) == va.VARLEN_ERR_STRIDE
    assert _rotary(va, sq=(256, 0)) in _runs(va)  # one head read as many
    assert _rotary(va, sqo=(256, 0)) == _rotary(va, sqo=(128, 64)) == va.VARLEN_ERR_STRIDE  # heads and rows on one another
    # in place: the same strides, or none that matter
    assert _rotary(va, qo=0x1000) in _runs(va)
    assert _rotary(va, qo=0x1000, sqo=(512, 64)) == _rotary(va, qo=0x1000, sq=(64, 640), sqo=(256, 64)) == va.VARLEN_ERR_STRIDE
    assert _rotary(va, ko=0x2000, sko=(512, 64), total=1) in _runs(va)


def test_rotary_cache_write_refusals(va):
    for kind in (0, 1):
        assert _write(va, _cache(va, type=kind)) in _runs(va)
    assert _write(va, _cache(va, block_table=None, seqlens=None, max_pages=-1)) in _runs(va)  # not looked at
    assert _write(va, c=0) == _write(va, rope=0) == va.VARLEN_ERR_NULL
    for name in ("q", "k", "v", "pos", "slots", "qo"):
        assert _write(va, **{name: None}) == va.VARLEN_ERR_NULL
    assert _write(va, slots=0x204) == _write(va, v=0x2808) == va.VARLEN_ERR_ALIGN
    assert _write(va, q=None, qo=None, heads=0) in _runs(va)
    assert _write(va, heads=-1) == _write(va, total=-1) == _write(va, heads=1 << 20) == va.VARLEN_ERR_SHAPE
    assert _write(va, st=(128, 60)) == _write(va, sqo=(256, 0)) == _write(va, qo=0x1000, sqo=(512, 64)) == va.VARLEN_ERR_STRIDE
    assert _write(va, _cache(va, num_pages=0)) == va.VARLEN_ERR_SHAPE
    assert _write(va, pos=None, slots=None, total=0) in _runs(va)


def test_tree_refusals(va):
    c = _cache(va)
    r, S = ctypes.byref(c), va.VarlenStride

    def call(masks=0x500, words=1, pos=None, left=-1, total=10, heads=4, scale=0.125, lse=0x3000, ws=0x100000, nb=1 << 40):
        return va.LIB.varlen_attn_fwd_paged_tree(0x1000, S(256, 64), 0x2000, 1, total, heads, 0, r, scale, masks, words, pos, left,
                                                 0x1000, S(256, 64), lse, ws, nb, None)

    assert call() in _runs(va) and call(pos=0x600, left=5) in _runs(va) and call(words=1 << 20) in _runs(va)
    assert call(masks=None) == call(left=0) == call(lse=None) == va.VARLEN_ERR_NULL
    for words in (0, -1, (1 << 20) + 1):
        assert call(words=words) == va.VARLEN_ERR_SHAPE
    assert call(heads=3) == call(scale=0.0) == call(total=-1) == va.VARLEN_ERR_SHAPE
    assert call(masks=0x502) == call(pos=0x602, left=5) == va.VARLEN_ERR_ALIGN
    assert call(nb=0) == call(ws=None) == va.VARLEN_ERR_WORKSPACE


def test_turns(va):
    """Frequencies in radians a position as whole 2^-64 turns: within 2^-52 turn relative to f / 2 pi and of one unit."""
    freq = [1.0, 0.0, 1e-4, 2 * math.pi, -1.0, 100.0, 1e-30, -1e-30]
    st, turns = va.varlen_attn_rotary_turns(freq)
    assert st == 0 and turns[1] == 0
    for f, t in zip(freq, turns):
        want = (f / (2 * math.pi)) % 1.0
        d = abs(t / 2 ** 64 - want)
        assert min(d, 1 - d) <= 2.0 ** -52 * max(1.0, abs(f) / (2 * math.pi)) + 2.0 ** -64
    for bad in (math.inf, math.nan):
        assert va.varlen_attn_rotary_turns([1.0, bad])[0] == va.VARLEN_ERR_SHAPE
    assert va.LIB.varlen_attn_rotary_turns(None, 1, None) == va.VARLEN_ERR_NULL
    assert va.LIB.varlen_attn_rotary_turns(None, 0, None) == 0
    assert va.LIB.varlen_attn_rotary_turns(None, -1, None) == va.VARLEN_ERR_SHAPE


def test_frequencies(va):
    f, s = va.rotary_frequencies(64)
    assert s == 1.0 and f.dtype == torch.float64 and torch.equal(f, 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64))
    f4, s = va.rotary_frequencies(64, stretch=4.0, how="linear")
    assert s == 1.0 and torch.equal(f4, f / 4)
    f4, s = va.rotary_frequencies(64, stretch=4.0, how="base")
    assert s == 1.0 and f4[0] == 1.0 and abs(f4[-1] / f[-1] - 0.25) < 1e-12
    f4, s = va.rotary_frequencies(64, stretch=4.0, trained=4096)
    turns = f * 4096 / (2 * math.pi)
    assert abs(s - (0.1 * math.log(4) + 1)) < 1e-15
    assert torch.equal(f4[turns >= 32], f[turns >= 32]) and torch.allclose(f4[turns <= 1], f[turns <= 1] / 4, rtol=1e-15)
    assert ((f4 <= f) & (f4 >= f / 4 * (1 - 1e-15))).all()
    for kw in ({"rotary_dim": 7}, {"rotary_dim": 0}, {"rotary_dim": 8, "base": 0.0}, {"rotary_dim": 8, "stretch": -1.0},
               {"rotary_dim": 8, "how": "other"}):
        with pytest.raises(ValueError):
            va.rotary_frequencies(**kw)


# ------------------------------------------------------------------ the binding

def test_pool_binding(va):
    table, lens, free, count = (torch.zeros(s, dtype=torch.int32) for s in ((3, 4), (3,), (9,), (1,)))
    pool = va.PagePool(table, lens, free, count, 16)
    assert pool.struct.seqlens == pool.struct.seqlens_out == lens.data_ptr() and pool.struct.num_pages == 9
    with pytest.raises(AttributeError):
        pool.seqlens = lens.clone()
    pool.seqlens += 1  # the same tensor
    for bad in ((table.long(), lens, free, count), (table[:, ::2], lens, free, count), (table, lens[:2], free, count),
                (table, lens, free.long(), count), (table, lens, free[::2], count), (table, lens, free, torch.zeros(2, dtype=torch.int32)),
                (table, lens.long(), free, count)):
        with pytest.raises(ValueError):
            va.PagePool(*bad, 16)
    for more in ((lens.clone()[:2], None), (None, count.long())):
        with pytest.raises(ValueError):
            va.PagePool(table, lens, free, count, 16, *more)


def test_step_binding(va):
    table, lens, free, count = (torch.zeros(s, dtype=torch.int32) for s in ((3, 4), (3,), (9,), (1,)))
    pool = va.PagePool(table, lens, free, count, 16)
    plan = va.StepPlan(3, 10, "cpu")
    assert plan.masks is None and plan.slots.dtype == torch.int64
    with pytest.raises(AttributeError):
        plan.slots = plan.slots.clone()
    for call in (lambda: va.cache_plan(pool, va.StepPlan(2, 10, "cpu"), lens),
                 lambda: va.cache_plan(pool, plan, lens, parents=torch.zeros(10, dtype=torch.int32)),  # no masks
                 lambda: va.cache_plan(pool, va.StepPlan(3, 10, "cpu", mask_words=1), lens, parents=torch.zeros(9, dtype=torch.int32)),
                 lambda: va.cache_plan(pool, plan, lens.long()), lambda: va.cache_plan(pool, plan, lens[:2]),
                 lambda: va.cache_trim(pool, lens[:2]), lambda: va.cache_trim(pool, lens, torch.zeros(3, dtype=torch.int32)),
                 lambda: va.cache_plan(pool, plan, lens)):  # on the CPU
        with pytest.raises(ValueError):
            call()


def test_rotary_binding(va):
    rope = va.Rotary([1.0, 0.5, 0.25, 0.125], device="cpu")
    assert rope.rotary_dim == 8 and rope.struct.rotary_dim == 8 and rope.turns.dtype == torch.int64
    with pytest.raises(AttributeError):
        rope.turns = rope.turns.clone()
    with pytest.raises(va.VarlenError):
        va.Rotary([math.inf] * 4, device="cpu")
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(5, dtype=torch.int32)
    for call in (lambda: va.rotary(q, k, rope), lambda: va.rotary(q.float(), k, rope, pos), lambda: va.rotary(q, k[:4], rope, pos),
                 lambda: va.rotary(q, k[..., ::2], rope, pos), lambda: va.rotary(q, k, rope, pos.long()),
                 lambda: va.rotary(q, k, rope, pos[:4]), lambda: va.rotary(q, k, rope, pos, q_out=k),
                 lambda: va.rotary(q, k, rope, cu_seqlens=pos.long()), lambda: va.rotary(q, k, rope, pos)):  # on the CPU
        with pytest.raises(ValueError):
            call()
    cache = va.PagedCache(**_tensors())
    slots = torch.zeros(5, dtype=torch.int64)
    for call in (lambda: va.rotary_cache_write(cache, q, k[:, :1], k, rope, pos, slots),
                 lambda: va.rotary_cache_write(cache, q, k, k, rope, pos, pos), lambda: va.rotary_cache_write(cache, q[:4], k, k, rope, pos, slots),
                 lambda: va.rotary_cache_write(cache, q, k, k, rope, pos, slots, q_out=k), lambda: va.rotary_cache_write(cache, q, k, k, rope, pos, slots)):
        with pytest.raises(ValueError):
            call()


def test_tree_and_move_binding(va):
    cache = va.PagedCache(**_tensors())
    q, cu = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    masks, pos = torch.zeros(5, 1, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    tree = va.attention_fwd_paged_tree
    for call in (lambda: tree(q, cache, cu, masks.long()), lambda: tree(q, cache, cu, masks[:4]), lambda: tree(q, cache, cu, masks[:, 0]),
                 lambda: tree(q, cache, cu[:3], masks), lambda: tree(q, cache, cu, masks, positions=pos.long()),
                 lambda: tree(q, cache, cu, masks, positions=pos[:4]), lambda: tree(q, cache, cu, torch.zeros(5, 4, dtype=torch.int32)[:, ::2]),
                 lambda: tree(q, cache, cu, masks, lse=torch.zeros(5, 4)), lambda: tree(q, cache, cu, masks, out=q[:, :2]),
                 lambda: tree(q, cache, cu, masks)):  # on the CPU
        with pytest.raises(ValueError):
            call()
    kept, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: va.cache_move(cache, cu, kept.long(), lens), lambda: va.cache_move(cache, cu, kept[:2], lens),
                 lambda: va.cache_move(cache, cu, kept.T.contiguous().T, lens), lambda: va.cache_move(cache, cu, kept, lens[:2]),
                 lambda: va.cache_move(cache, cu[:2], kept, lens), lambda: va.cache_move([cache, cache], cu, kept, lens)):
        with pytest.raises(ValueError):
            call()
    assert va.cache_move([], cu, kept, lens) is None
