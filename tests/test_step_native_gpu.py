"""The calls around a step through the native binding and through ctypes: the same bits, the same errors."""
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
    assert varlen_attn.NATIVE is not None, "the native binding is not built"
    return varlen_attn


class Watched:
    """The native binding, counting the calls that it answers and those that it leaves to ctypes."""

    def __init__(self, native):
        self.native, self.answered, self.left = native, 0, 0

    def __getattr__(self, name):
        f = getattr(self.native, name)

        def call(*a):
            got = f(*a)
            if got is NotImplemented:
                self.left += 1
            else:
                self.answered += 1
            return got
        return call


def _ways(va, monkeypatch, run, native=True):
    """run() by each way: equal bits; `native`: whether the binding has to have taken the calls, or left them."""
    w = Watched(va.NATIVE)
    got = []
    for how in (w, None):
        with monkeypatch.context() as m:
            m.setattr(va, "NATIVE", how)
            got.append([None if t is None else t.clone() for t in run()])
    torch.cuda.synchronize()
    assert (w.answered > 0 and w.left == 0) if native else (w.answered == 0 and w.left > 0)
    for a, b in zip(*got, strict=True):
        assert (a is None) == (b is None)
        if a is not None:
            assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride() and a.device == b.device
            assert a.requires_grad == b.requires_grad
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _rows(n, heads, dim, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.full((n, heads, dim + pad), math.nan, dtype=torch.bfloat16)
    x[..., :dim] = torch.randn(n, heads, dim, generator=g).to(torch.bfloat16)
    return x.to(DEV)[..., :dim]


def _step(va, kind="bf16", dim=64, heads=4, kv=2, new=(3, 0, 40), lens=(20, 5, 300), page=16, words=2, extra=2):
    """A cache that holds a step's rows, and that step's inputs."""
    total = sum(new) + extra
    cache, _, _ = C.make_cache(lens, kv, dim, page, kind, DEV, seed=1)
    g = torch.Generator().manual_seed(2)
    parents = [p for n in new for p in S.random_tree(n, g)] + [0] * extra
    pos = [n - m + i for n, m in zip(lens, new) for i in range(m)] + [0] * extra
    rows, masks = [S.ancestors(parents[a:a + n]) for a, n in zip([sum(new[:i]) for i in range(len(new))], new)], None
    masks = torch.cat([S.pack(r, words) for r in rows if len(r)] + [torch.zeros(extra, words, dtype=torch.int32)]).to(DEV)
    return dict(cache=cache, total=total, new=list(new), parents=_ints(parents), pos=_ints(pos), cu=C.cu_of(new, DEV), masks=masks,
                q=_rows(total, heads, dim, 3), k=_rows(total, kv, dim, 4, pad=16), v=_rows(total, kv, dim, 5), lens=list(lens), page=page)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,heads,kv", [(64, 4, 2), (96, 1, 1), (128, 7, 7)])
def test_same_bits(va, monkeypatch, kind, dim, heads, kv):
    s = _step(va, kind, dim, heads, kv)
    rope = va.Rotary(va.rotary_frequencies(dim)[0], device=DEV)
    q, k, v, cache = s["q"], s["k"], s["v"], s["cache"]
    _ways(va, monkeypatch, lambda: va.rotary(q, k, rope, s["pos"]))
    _ways(va, monkeypatch, lambda: va.rotary(q, None, rope, positions=s["pos"], cu_seqlens=s["pos"].long()))  # positions go first
    _ways(va, monkeypatch, lambda: [t[:sum(s["new"])] for t in va.rotary_bwd(q, k, rope, cu_seqlens=s["cu"])])
    _ways(va, monkeypatch, lambda: va.rotary(q, k, rope, s["pos"], q_out=torch.zeros_like(q), k_out=torch.zeros_like(v)))
    table = cache.block_table.tolist()
    slots = [table[b][p // s["page"]] * s["page"] + p % s["page"] for b, n in enumerate(s["new"]) for p in
             range(s["lens"][b] - n, s["lens"][b])] + [-1, -1]

    def write(queries, out):
        for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale):
            if t is not None:
                t.view(torch.uint8).fill_(0x21)
        turned = va.rotary_cache_write(cache, queries, k, v, rope, s["pos"], _ints(slots, torch.int64), q_out=out)
        return [turned, cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale]
    _ways(va, monkeypatch, lambda: write(q, None))
    _ways(va, monkeypatch, lambda: write(q, torch.zeros_like(q)))
    _ways(va, monkeypatch, lambda: write(None, None))
    for more in ({}, {"scale": 0.3}, {"window_left": 30, "positions": s["pos"]}, {"max_seqlen_q": 40}, {"window_left": -7}):
        _ways(va, monkeypatch, lambda: [t[:, :sum(s["new"])] if t.dim() == 2 else t[:sum(s["new"])] for t in
                                        va.attention_fwd_paged_tree(q, cache, s["cu"], s["masks"], **more)])
    assert va.varlen_attn_get_device_status() == 0


@pytest.mark.parametrize("trees", [False, True])
def test_same_plans(va, monkeypatch, trees):
    new, old, page = [3, 0, 40], [13, 5, 260], 16
    total = sum(new) + 2
    need = [-(-n // page) for n in old]
    parents = _ints([-1, 0, 0] + list(range(-1, 39)) + [0, 0])

    def run():
        table = _ints([list(range(i * 20, i * 20 + n)) + [0] * (20 - n) for i, n in enumerate(need)])
        pool = va.PagePool(table, _ints(old), _ints(list(range(60, 80)) + [0] * 60), _ints([20]), page)  # 80 pages, 20 of them free
        plan = va.StepPlan(3, total, DEV, mask_words=2 if trees else 0)
        va.cache_plan(pool, plan, _ints(new), parents=parents if trees else None)
        between = [plan.cu_seqlens, plan.slots, plan.positions, plan.unplaced, plan.masks] + [t.clone() for t in (pool.seqlens, pool.free_count)]
        va.cache_trim(pool, _ints([1, 0, 9]), plan.cu_seqlens)
        va.cache_trim(pool, _ints([1000, 2, 40]))
        return between + [pool.block_table, pool.seqlens, pool.free_pages, pool.free_count]
    _ways(va, monkeypatch, run)
    assert va.varlen_attn_get_device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("layers", [1, 3])
def test_same_moves(va, monkeypatch, kind, layers):
    new, lens = [5, 0, 30], [20, 5, 300]
    kept = torch.zeros(3, 9, dtype=torch.int32, device=DEV)[:, :4]
    kept.copy_(_ints([[1, 3, 4, 0], [0] * 4, [0, 7, 8, 29]]))

    def run():
        made = [C.make_cache(lens, 2, 64, 16, kind, DEV, seed=i)[0] for i in range(layers)]
        caches = made[:1] + [va.PagedCache(c.k_pages, c.v_pages, made[0].block_table, made[0].seqlens, c.k_scale, c.v_scale)
                             for c in made[1:]]  # one table
        va.cache_move(caches if layers > 1 else caches[0], C.cu_of(new, DEV), kept, _ints([3, 0, 4]))
        return [t for c in caches for t in (c.k_pages, c.v_pages, c.k_scale, c.v_scale)]
    _ways(va, monkeypatch, run)
    assert va.varlen_attn_get_device_status() == 0


def test_a_side_stream_that_is_current(va, monkeypatch):
    """Current: the binding takes it.  Named: ctypes does."""
    s = _step(va)
    rope = va.Rotary(va.rotary_frequencies(64)[0], device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()

    def run():
        with torch.cuda.stream(side):
            x = s["q"] * 2  # what the call waits for on this stream
            got = va.rotary(x, s["k"], rope, s["pos"]) + va.attention_fwd_paged_tree(x, s["cache"], s["cu"], s["masks"])
            n = sum(s["new"])
            got = [got[0], got[1], got[2][:n], got[3][:, :n]]
        side.synchronize()
        return got
    _ways(va, monkeypatch, run)
    w = Watched(va.NATIVE)
    monkeypatch.setattr(va, "NATIVE", w)
    a = va.rotary(s["q"], s["k"], rope, s["pos"], stream=side)
    side.synchronize()
    assert w.answered == w.left == 0
    assert torch.equal(a[0], va.rotary(s["q"], s["k"], rope, s["pos"])[0]) and w.answered == 1


def test_inputs_with_gradients_and_subclasses(va, monkeypatch):
    s = _step(va)
    rope = va.Rotary(va.rotary_frequencies(64)[0], device=DEV)
    leaf = torch.nn.Parameter(s["q"].clone())
    _ways(va, monkeypatch, lambda: va.rotary(leaf, s["k"], rope, s["pos"]))
    with torch.inference_mode():
        _ways(va, monkeypatch, lambda: va.rotary(s["q"], s["k"], rope, s["pos"]))


def test_what_the_binding_leaves_to_ctypes(va, monkeypatch):
    """Whole numbers as scale, unsigned masks: answered, by ctypes."""
    s = _step(va)
    n = sum(s["new"])
    for more in ({"scale": 1}, {"masks": s["masks"].view(torch.uint32)}):
        args = {"masks": s["masks"], **more}
        _ways(va, monkeypatch, lambda: [t[:n] if t.dim() == 3 else t[:, :n] for t in
                                        va.attention_fwd_paged_tree(s["q"], s["cache"], s["cu"], **args)], native=False)


def test_refusals_are_the_same(va, monkeypatch):
    s = _step(va)
    q, k, v, cache, pos, cu, masks = (s[x] for x in ("q", "k", "v", "cache", "pos", "cu", "masks"))
    rope = va.Rotary(va.rotary_frequencies(64)[0], device=DEV)
    wide = va.Rotary(va.rotary_frequencies(128)[0], device=DEV)
    far = va.Rotary(va.rotary_frequencies(64)[0], device="cpu")
    slots = torch.full((s["total"],), -1, dtype=torch.int64, device=DEV)
    odd = torch.zeros(s["total"] * 4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(-1, 4, 64)  # 2 bytes off
    table, lens, free, count = _ints([[0] * 4] * 3), _ints([0] * 3), _ints([0] * 9), _ints([9])
    pool, plan = va.PagePool(table, lens, free, count, 16), va.StepPlan(3, 10, DEV, mask_words=1)
    low = va.PagePool(table, lens, free, count, 0)  # pages of no rows: the library's refusal
    kept = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    calls = [lambda: va.rotary(q, k, rope), lambda: va.rotary(q.float(), k, rope, pos), lambda: va.rotary(q, k[:4], rope, pos),
             lambda: va.rotary(q, k[..., ::2], rope, pos), lambda: va.rotary(q, k, rope, pos.long()),
             lambda: va.rotary(q, k, rope, pos.cpu()), lambda: va.rotary(q.cpu(), k, rope, pos), lambda: va.rotary(q, k, far, pos),
             lambda: va.rotary(q, k, rope, pos, q_out=k), lambda: va.rotary(q, k, rope, cu_seqlens=pos.long()),
             lambda: va.rotary(odd, k, rope, pos), lambda: va.rotary(q, k, wide, pos), lambda: va.rotary(None, k, rope, pos),
             lambda: va.rotary(q, k, rope, cu_seqlens=pos[:0]), lambda: va.rotary(q, k, rope, pos, q_out=q[:, :1].expand(-1, 4, -1)),
             lambda: va.rotary_cache_write(cache, q, k[:, :1], k, rope, pos, slots),
             lambda: va.rotary_cache_write(cache, q, k, k, rope, pos, pos), lambda: va.rotary_cache_write(cache, q, k, v, far, pos, slots),
             lambda: va.rotary_cache_write(cache, odd, k, v, rope, pos, slots), lambda: va.rotary_cache_write(cache, q, k, v, wide, pos, slots),
             lambda: va.rotary_cache_write(cache, q, k, v, rope, pos, slots, q_out=k), lambda: va.rotary_cache_write(cache, q, None, v, rope, pos, slots),
             lambda: va.cache_plan(pool, va.StepPlan(2, 10, DEV), lens), lambda: va.cache_plan(pool, plan, lens.long()),
             lambda: va.cache_plan(pool, plan, lens, parents=lens), lambda: va.cache_plan(pool, plan, lens.cpu()),
             lambda: va.cache_plan(low, plan, lens), lambda: va.cache_trim(low, lens), lambda: va.cache_trim(pool, lens[:2]),
             lambda: va.cache_trim(pool, lens, lens), lambda: va.cache_move(cache, cu, kept.long(), lens),
             lambda: va.cache_move([cache, cache], cu, kept[:2], lens), lambda: va.cache_move(cache, cu, kept, lens[:2]),
             lambda: va.cache_move(cache, cu.cpu(), kept, lens), lambda: va.cache_move(cache, cu, kept.T.contiguous().T, lens),
             lambda: va.attention_fwd_paged_tree(q, cache, cu, masks.long()), lambda: va.attention_fwd_paged_tree(q, cache, cu, masks[:4]),
             lambda: va.attention_fwd_paged_tree(q[:, :3], cache, cu, masks), lambda: va.attention_fwd_paged_tree(odd, cache, cu, masks),
             lambda: va.attention_fwd_paged_tree(q, cache, cu, masks, scale=0.0),
             lambda: va.attention_fwd_paged_tree(q, cache, cu, masks, window_left=3, positions=pos[:4]),
             lambda: va.attention_fwd_paged_tree(q, cache, cu[:3], masks)]
    kinds = set()
    for i, call in enumerate(calls):
        said = []
        for how in (va.NATIVE, None):
            with monkeypatch.context() as m:
                m.setattr(va, "NATIVE", how)
                with pytest.raises(Exception) as e:
                    call()
                said.append((e.type, str(e.value)))
        assert said[0] == said[1], i
        kinds.add(said[0][0])
    assert kinds >= {ValueError, va.VarlenError}
    torch.cuda.synchronize()
    assert va.varlen_attn_get_device_status() == 0


def test_windows_past_32_bits(va, monkeypatch):
    s = _step(va)
    n = sum(s["new"])
    want = va.attention_fwd_paged_tree(s["q"], s["cache"], s["cu"], s["masks"])
    for how in (va.NATIVE, None):
        monkeypatch.setattr(va, "NATIVE", how)
        for left in ((1 << 31) - 1, 1 << 31, (1 << 32) + 5, 1 << 80):
            got = va.attention_fwd_paged_tree(s["q"], s["cache"], s["cu"], s["masks"], window_left=left, positions=s["pos"])
            assert torch.equal(got[0][:n], want[0][:n]) and torch.equal(got[1][:, :n], want[1][:, :n])
    torch.cuda.synchronize()
    assert va.varlen_attn_get_device_status() == 0


def test_threads_on_their_own_streams(va):
    """Calls of four threads at once, each on a stream that is current in its thread: the bits of one alone."""
    import threading
    s = _step(va)
    n = sum(s["new"])
    rope = va.Rotary(va.rotary_frequencies(64)[0], device=DEV)

    def run(q):
        got = va.rotary(q, s["k"], rope, s["pos"]) + va.attention_fwd_paged_tree(q, s["cache"], s["cu"], s["masks"])
        return [got[0], got[1], got[2][:n], got[3][:, :n]]
    qs = [s["q"] * f for f in (1, 0.5, 2, -1)]
    want = [run(q) for q in qs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = run(qs[i])
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i], strict=True)):
                        wrong.append(i)
        except Exception as e:
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not wrong and not any(t.is_alive() for t in threads)
    assert va.varlen_attn_get_device_status() == 0
