"""The paged cache and the attention over it against plain 64-bit forms, on a
GPU: writing, reading back, attention over pages, and the three together, for
both cache types, all head sizes, grouped heads, page sizes, bands, layouts
and the sizes where tiles, pages and segments end inside one another."""
import math

import pytest
import torch

from tests import paged_cases as C

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def va():
    from packed_variable_length_varlen_gb300 import varlen_attn
    return varlen_attn


def _ok(va):
    st = va.varlen_attn_get_device_status()
    assert st == 0, va.varlen_attn_status_string(st)


def _q(total, heads, dim, seed=1, amp=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(total, heads, dim, generator=g) * amp).to(torch.bfloat16).to(DEV)
    if not pad:
        return q
    wide = torch.full((total, heads, dim + pad), math.nan, dtype=torch.bfloat16, device=DEV)
    wide[..., :dim] = q
    return wide[..., :dim]


def _attend(va, new, lens, heads, kv, dim, page, kind, causal=False, window=(-1, -1), order="nhd", hint=None, seed=0,
            amp=1.0, extra=0, pad=0, fill=None, columns=1):
    """Runs the attention, checks it; returns (out, lse)."""
    cache, k, v = C.make_cache(lens, kv, dim, page, kind, DEV, seed=seed, order=order, amp=amp, fill=fill,
                               columns=columns)
    total = sum(new) + extra
    q = _q(total, heads, dim, seed=seed + 1, amp=amp, pad=pad)
    cu = C.cu_of(new, DEV)
    out = torch.full((total, heads, dim + pad), 77.0, dtype=torch.bfloat16, device=DEV)[..., :dim]
    lse = torch.full((heads, total), 77.0, device=DEV)
    va.attention_fwd_paged(q, cache, cu, max_seqlen_q=max(new) if hint is None else hint, out=out, lse=lse,
                           causal=causal, window=window)
    _ok(va)
    left, right = window
    if causal:
        right = 0
    scale = float(torch.tensor(dim ** -0.5, dtype=torch.float32))
    at = 0
    for b, n in enumerate(new):
        ref = C.attend(q[at:at + n], k[b], v[b], scale, left, right)
        C.check_attend(out[at:at + n], lse[:, at:at + n], ref, dim, lens[b])
        at += n
    assert (out[at:] == 77.0).all() and (lse[:, at:] == 77.0).all()  # rows behind the last segment stay
    if pad:
        whole = out.as_strided((total, heads, dim + pad), (heads * (dim + pad), dim + pad, 1))
        assert (whole[..., dim:] == 77.0).all()
    return out, lse


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("page,order", [(16, "nhd"), (64, "hnd"), (256, "padded"), (32, "together")])
def test_write_then_read(va, kind, dim, page, order):
    lens = [40, 0, 1, 17, 300, 16, 129]
    new = [7, 0, 1, 17, 130, 20, 0]  # the sixth brings more rows than its sequence holds: the first four drop
    heads = 3
    cache, k, v = C.make_cache(lens, heads, dim, page, kind, DEV, seed=5, order=order)
    before = [t.clone() for t in (cache.k_pages.contiguous().view(torch.uint8), cache.v_pages.contiguous().view(torch.uint8))]
    total = sum(new) + 5
    kn, vn = _q(total, heads, dim, 11, pad=32), _q(total, heads, dim, 12)
    cu = C.cu_of(new, DEV)
    va.cache_write(cache, kn, vn, cu)
    _ok(va)
    # what each place has to hold: the old rows with the new ones in their places
    at = 0
    touched = torch.zeros(before[0].shape[:2], dtype=torch.bool, device=DEV)
    for b, n in enumerate(new):
        for i, (x, held) in enumerate(((kn, k), (vn, v))):
            rows = x[at:at + n]
            first = lens[b] - n
            rows = rows[max(0, -first):]
            pos = torch.arange(max(first, 0), lens[b], device=DEV)
            pg = cache.block_table[b].long()[pos // page]
            touched[pg, pos % page] = True
            if kind == "bf16":
                held[b][pos] = rows.double()
                assert torch.equal((cache.k_pages if i == 0 else cache.v_pages)[pg, pos % page], rows)
            else:
                codes, s = C.quantise(rows)
                held[b][pos] = codes.double() * s.double()[..., None]
                got = (cache.k_pages if i == 0 else cache.v_pages).view(torch.uint8)[pg, pos % page]
                assert torch.equal(got, codes.view(torch.uint8))
                assert torch.equal((cache.k_scale if i == 0 else cache.v_scale)[pg, :, pos % page], s)
        at += n
    for pool, old in ((cache.k_pages, before[0]), (cache.v_pages, before[1])):
        assert torch.equal(pool.contiguous().view(torch.uint8)[~touched], old[~touched])
    # everything back, and a request for more rows than there are: zeros in front
    ask = [n + 2 for n in lens]
    ko = torch.full((sum(ask) + 3, heads, dim), 5.0, dtype=torch.bfloat16, device=DEV)
    vo = torch.full((sum(ask) + 3, heads, dim + 8), 5.0, dtype=torch.bfloat16, device=DEV)[..., :dim]
    va.cache_read(cache, C.cu_of(ask, DEV), sum(ask) + 3, ko, vo)
    _ok(va)
    at = 0
    for b, n in enumerate(ask):
        for o, held in ((ko, k), (vo, v)):
            assert (o[at:at + 2] == 0).all()
            assert torch.equal(o[at + 2:at + n], held[b].to(torch.bfloat16))
        at += n
    assert (ko[at:] == 5.0).all() and (vo[at:] == 5.0).all()


def test_write_e4m3_values(va):
    """Zeros, signed zeros, the borders of the scale, subnormal and largest values, infinities, NaN."""
    dim, heads = 64, 1
    rows = torch.zeros(12, dim)
    rows[1, 3] = 448.0
    rows[2, 3] = 450.0                    # the next bf16 above 448: the scale doubles
    rows[3, 0], rows[3, 1] = 2.0 ** -133, -(2.0 ** -130)
    rows[4, 5] = 3.3895e38
    rows[5, 5], rows[5, 6] = math.inf, 1.0
    rows[6, 7] = math.nan
    rows[7, :] = -0.0
    rows[8, 0], rows[8, 1] = 2.0 ** -120, 1.75 * 2.0 ** -119  # a scale at its least value
    rows[9] = torch.linspace(-448, 448, dim)
    rows[10] = torch.linspace(-1, 1, dim) * 2.0 ** 100
    rows[11, 2], rows[11, 3] = -math.inf, math.nan
    x = rows.to(torch.bfloat16)[:, None].to(DEV)
    cache, _, _ = C.make_cache([12], heads, dim, 16, "e4m3", DEV)
    va.cache_write(cache, x, x, C.cu_of([12], DEV))
    _ok(va)
    codes, s = C.quantise(x)
    pg = int(cache.block_table[0, 0])
    assert torch.equal(cache.k_pages.view(torch.uint8)[pg, :12], codes.view(torch.uint8))
    assert torch.equal(cache.v_pages.view(torch.uint8)[pg, :12], codes.view(torch.uint8))
    for got in (cache.k_scale[pg, :, :12].T, cache.v_scale[pg, :, :12].T):
        assert torch.equal(torch.isnan(got), torch.isnan(s))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(s))
    k, v = va.cache_read(cache, C.cu_of([12], DEV), 12)
    want = (codes.float() * s.float()[..., None]).to(torch.bfloat16)
    for got in (k, v):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_every_code_reads_back(va, kind):
    """All 254 finite codes at scales across the range, through the read and through a one-key attention
    (O = v exactly when a row sees one key)."""
    dim, page, heads = 128, 16, 2
    lens = [1] * 24
    cache, _, _ = C.make_cache(lens, heads, dim, page, "e4m3" if kind == "e4m3" else "bf16", DEV)
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    codes[127], codes[255] = 0, 0
    exps = [-115, -100, -64, -33, -20, -17, -12, -10, -8, -6, -4, -2, -1, 0, 1, 2, 4, 6, 7, 8, 20, 60, 100, 119]
    want = []
    for b, e in enumerate(exps):
        pg = int(cache.block_table[b, 0])
        val = codes.view(torch.float8_e4m3fn).reshape(heads, dim).double() * 2.0 ** e
        if kind == "e4m3":
            for pool, sc in ((cache.k_pages, cache.k_scale), (cache.v_pages, cache.v_scale)):
                pool.view(torch.uint8)[pg, 0] = codes.reshape(heads, dim)
                sc[pg, :, 0] = 2.0 ** e
        else:
            cache.k_pages[pg, 0] = val.to(torch.bfloat16)
            cache.v_pages[pg, 0] = val.to(torch.bfloat16)
        want.append(val.to(torch.bfloat16))
    want = torch.stack(want)
    cu = C.cu_of(lens, DEV)
    k, v = va.cache_read(cache, cu, len(lens))
    assert torch.equal(k, want) and torch.equal(v, want)
    q = torch.zeros(len(lens), heads * 2, dim, dtype=torch.bfloat16, device=DEV)
    for hint in (1, 0):
        out, lse = va.attention_fwd_paged(q, cache, cu, max_seqlen_q=hint)
        _ok(va)
        assert torch.equal(out, want.repeat_interleave(2, 1))
        assert (lse == 0).all()


# ------------------------------------------------------------------ attention

NEW = [1, 0, 1, 3, 1, 16, 1, 5, 2, 9]
LENS = [5, 7, 0, 200, 64, 16, 700, 3, 129, 65]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("heads,kv,page", [(2, 2, 16), (4, 1, 64), (6, 2, 128), (14, 2, 32), (16, 1, 256)])
@pytest.mark.parametrize("causal,window", [(False, (-1, -1)), (True, (-1, -1)), (True, (37, -1))])
def test_few_rows(va, kind, dim, heads, kv, page, causal, window):
    """Single and drafted tokens: segments of up to 16 rows, caches empty, shorter than the queries, and longer."""
    _attend(va, NEW, LENS, heads, kv, dim, page, kind, causal, window)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("heads,kv,page", [(2, 2, 16), (8, 2, 64), (7, 1, 32), (3, 1, 1024)])
@pytest.mark.parametrize("causal,window", [(False, (-1, -1)), (True, (-1, -1)), (False, (100, 20)), (False, (0, 0))])
def test_chunks(va, kind, dim, heads, kv, page, causal, window):
    """Chunks beside single tokens: lengths around the tile sizes, more queries than keys, empty segments."""
    _attend(va, [130, 1, 0, 257, 64, 65, 33, 300], [700, 300, 40, 257, 128, 1000, 20, 256], heads, kv, dim, page,
            kind, causal, window)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("order", ["hnd", "padded", "together"])
def test_layouts(va, kind, order):
    """Pages in head-major order, with padding, and K beside V; padded query and output rows; rows behind the last."""
    _attend(va, [3, 150, 1], [90, 400, 257], 8, 2, 96, 32, kind, True, order=order, pad=8, extra=9)
    _attend(va, [3, 1, 1], [90, 400, 257], 8, 2, 128, 64, kind, True, order=order, pad=16, extra=3)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1], [4], [40], [300]])
def test_long_cache(va, kind, new):
    """One long sequence that many CTAs share, and its join."""
    _attend(va, new, [20011], 8, 2, 128, 64, kind, True)
    _attend(va, new, [20011], 8, 2, 64, 16, kind, True, (5000, -1))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_many_sequences(va, kind):
    """More sequences than a CTA has threads, most of them short, some empty."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 120, (700,), generator=g).tolist()
    new = [int(torch.randint(0, 3, (1,), generator=g)) for _ in lens]
    _attend(va, new, lens, 4, 2, 64, 16, kind, True)
    new[350] = 180
    lens[350] = 900
    _attend(va, new, lens, 4, 2, 64, 16, kind, True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,kv", [(128, 1), (56, 1), (40, 1), (56, 56), (5, 5)])
def test_head_groups(va, kind, heads, kv):
    _attend(va, [1, 3, 40], [100, 30, 300], heads, kv, 128, 32, kind, True)
    _attend(va, [1, 2, 1], [100, 30, 300], heads, kv, 64, 32, kind, True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hint", [0, 1, 2, 1000000])
def test_the_hint_is_only_a_hint(va, kind, hint):
    _attend(va, [1, 200, 7], [300, 800, 64], 4, 2, 128, 64, kind, True, hint=hint)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 2], [100, 300]])
def test_growing_scores(va, kind, new):
    """Key sizes that grow along the cache, so that the running maximum moves again and again, and large scores."""
    def fill(x, b, i):
        if i == 1:
            return x
        ramp = torch.linspace(0.01, 6.0, x.shape[0], device=x.device)[:, None, None]
        return (x.float() * ramp).to(torch.bfloat16)
    _attend(va, new, [900, 2000], 4, 2, 128, 64, kind, False, fill=fill, amp=2.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[2], [200]])
def test_small_and_large_values(va, kind, new):
    """Values near 2^40 and 2^-40 and keys of very different sizes: scales far from one."""
    def fill(x, b, i):
        e = torch.randint(-6, 3, x.shape[:2], generator=torch.Generator().manual_seed(7)).to(x.device)
        s = torch.exp2(e.float())[..., None] * (2.0 ** 40 if i == 1 else 1.0)
        s[::3] *= 2.0 ** -80 if i == 1 else 1.0
        return (x.float() * s).to(torch.bfloat16)
    _attend(va, new, [500], 4, 2, 128, 16, kind, True, fill=fill)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 100])
def test_unseen_rows_may_hold_anything(va, kind, n):
    """Positions left of every query's window hold NaN, in pages that the table still names."""
    left, ln = 50, 400

    def fill(x, b, i):
        x = x.clone()
        x[:ln - n - left] = math.nan
        return x
    cache, k, v = C.make_cache([ln], 2, 128, 16, kind, DEV, fill=fill)
    first = ln - n - left
    # and the pages wholly behind the window are gone
    cache.block_table[0, :first // 16] = -1
    q = _q(n, 4, 128)
    out, lse = va.attention_fwd_paged(q, cache, C.cu_of([n], DEV), max_seqlen_q=n, causal=True, window=(left, -1))
    _ok(va)
    k, v = k[0][first:], v[0][first:]
    ref = C.attend(q, k, v, float(torch.tensor(128 ** -0.5)), left, 0)
    C.check_attend(out, lse, ref, 128, ln)


def test_non_finite_vectors_show(va):
    """A NaN that is written is seen by the queries that see its key, in both cache types, and by no other segment."""
    for kind in ("bf16", "e4m3"):
        for n in (1, 150):
            cache, _, _ = C.make_cache([200, 200], 2, 64, 16, kind, DEV)
            k, v = _q(2 * n, 2, 64, 3), _q(2 * n, 2, 64, 4)
            v[0, 0, 5] = math.nan
            cu = C.cu_of([n, n], DEV)
            va.cache_write(cache, k, v, cu)
            out, _ = va.attention_fwd_paged(_q(2 * n, 4, 64), cache, cu, max_seqlen_q=n, causal=True)
            _ok(va)
            assert torch.isnan(out[:n, :2, 5]).all()
            assert torch.isfinite(out[:, 2:]).all() and torch.isfinite(out[n:]).all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prompt_then_tokens(va, kind):
    """A prompt written and attended in chunks, then tokens one by one: each step equals one call of the packed
    forward over the rows read back."""
    dim, heads, kv, page = 128, 4, 2, 16
    steps = [[100, 37], [64, 1], [1, 1], [1, 1], [3, 0]]
    total = [sum(s[b] for s in steps) for b in range(2)]
    cache, _, _ = C.make_cache(total, kv, dim, page, kind, DEV)
    cache.seqlens.zero_()
    for i, new in enumerate(steps):
        n, cu = sum(new), C.cu_of(new, DEV)
        cache.seqlens += torch.tensor(new, dtype=torch.int32, device=DEV)
        va.cache_write(cache, _q(n, kv, dim, 50 + i), _q(n, kv, dim, 60 + i), cu)
        q = _q(n, heads, dim, 70 + i)
        out, lse = va.attention_fwd_paged(q, cache, cu, max_seqlen_q=max(new), causal=True)
        held = cache.seqlens.tolist()
        cu_k = C.cu_of(held, DEV)
        k, v = va.cache_read(cache, cu_k, sum(held))
        rep = lambda t: t.repeat_interleave(heads // kv, 1).contiguous()  # noqa: E731
        o2, l2 = va.attention_fwd(q, rep(k), rep(v), cu, cu_k, causal=True)
        _ok(va)
        at = 0
        for b in range(2):
            ks, vs = k[cu_k[b]:cu_k[b + 1]].double(), v[cu_k[b]:cu_k[b + 1]].double()
            ref = C.attend(q[at:at + new[b]], ks, vs, float(torch.tensor(dim ** -0.5)), -1, 0)
            for o, l in ((out, lse), (o2, l2)):
                C.check_attend(o[at:at + new[b]], l[:, at:at + new[b]], ref, dim, held[b])
            at += new[b]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_and_replayed(va, kind):
    """Write and attention in one CUDA graph, replayed as the sequences grow; the captured lengths are device data."""
    dim, heads, kv, page = 64, 8, 2, 16
    cache, _, _ = C.make_cache([300, 150], kv, dim, page, kind, DEV)
    start = torch.tensor([200, 90], dtype=torch.int32, device=DEV)
    new = [1, 1]
    cu = C.cu_of(new, DEV)
    kn, vn, q = _q(2, kv, dim, 3), _q(2, kv, dim, 4), _q(2, heads, dim, 5)

    def step():
        cache.seqlens.add_(1)
        va.cache_write(cache, kn, vn, cu)
        return va.attention_fwd_paged(q, cache, cu, max_seqlen_q=1, causal=True)

    cache.seqlens.copy_(start)
    want = []
    for i in range(4):
        kn.copy_(_q(2, kv, dim, 30 + i))
        o, l = step()
        want.append((o.clone(), l.clone()))
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        o, l = step()
    torch.cuda.synchronize()
    cache.seqlens.copy_(start)
    for i in range(4):
        kn.copy_(_q(2, kv, dim, 30 + i))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])
    _ok(va)


def test_streams_and_repeats(va):
    """Two calls at once on two streams, each with its own workspace, give the bits of a call alone; so do repeats."""
    cache, _, _ = C.make_cache([5000, 3000], 2, 128, 64, "e4m3", DEV)
    cu = C.cu_of([40, 1], DEV)
    q = [_q(41, 8, 128, s) for s in (1, 2)]
    alone = [va.attention_fwd_paged(x, cache, cu, causal=True) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(5):
        got = [va.attention_fwd_paged(x, cache, cu, causal=True, stream=s) for x, s in zip(q, streams)]
        torch.cuda.synchronize()
        for (o, l), (o1, l1) in zip(alone, got):
            assert torch.equal(o, o1) and torch.equal(l, l1)
    _ok(va)


# ------------------------------------------------------------------ bad pages, far pages

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 90])
def test_bad_pages_are_reported(va, kind, n):
    """Entries that name no page: reads are zeros, writes drop, the status says so, and the next call is clean."""
    cache, k, v = C.make_cache([100, 100], 2, 64, 16, kind, DEV)
    good = cache.block_table.clone()
    bad = cache.k_pages.shape[0]
    cache.block_table[0, 3], cache.block_table[0, 4] = bad, -2147483648
    ko, vo = va.cache_read(cache, C.cu_of([100, 100], DEV), 200)
    assert va.varlen_attn_get_device_status() == va.VARLEN_ERR_DEVICE_BOUNDS
    hole = k[0].clone()
    hole[48:80] = 0
    assert torch.equal(ko[:100], hole.to(torch.bfloat16)) and torch.equal(ko[100:], k[1].to(torch.bfloat16))
    q, cu = _q(2 * n, 4, 64), C.cu_of([n, n], DEV)
    out, lse = va.attention_fwd_paged(q, cache, cu, max_seqlen_q=n, causal=True)
    assert va.varlen_attn_get_device_status() == va.VARLEN_ERR_DEVICE_BOUNDS
    vh = v[0].clone()
    vh[48:80] = 0
    for b, (kk, vv) in enumerate(((hole, vh), (k[1], v[1]))):
        ref = C.attend(q[b * n:(b + 1) * n], kk, vv, 0.125, -1, 0)
        C.check_attend(out[b * n:(b + 1) * n], lse[:, b * n:(b + 1) * n], ref, 64, 100)
    pools = [t.contiguous().view(torch.uint8).clone() for t in (cache.k_pages, cache.v_pages)]
    cache.block_table[0] = bad
    cache.block_table[1] = -1
    va.cache_write(cache, _q(200, 2, 64), _q(200, 2, 64), C.cu_of([100, 100], DEV))
    assert va.varlen_attn_get_device_status() == va.VARLEN_ERR_DEVICE_BOUNDS
    for t, old in zip((cache.k_pages, cache.v_pages), pools):
        assert torch.equal(t.contiguous().view(torch.uint8), old)
    cache.block_table.copy_(good)
    va.cache_read(cache, C.cu_of([100, 100], DEV), 200)
    _ok(va)


def test_lengths_past_the_table_are_clamped(va):
    """seqlens beyond what the table can name, and negative ones."""
    for n in (1, 100):
        cache, k, v = C.make_cache([160, 160], 2, 64, 16, "bf16", DEV)
        cache.seqlens.copy_(torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32))
        q, cu = _q(2 * n, 4, 64), C.cu_of([n, n], DEV)
        out, lse = va.attention_fwd_paged(q, cache, cu, max_seqlen_q=n, causal=True)
        _ok(va)
        ref = C.attend(q[:n], k[0], v[0], 0.125, -1, 0)
        C.check_attend(out[:n], lse[:, :n], ref, 64, 160)
        assert (out[n:] == 0).all() and (lse[:, n:] == -math.inf).all()
        ko, _ = va.cache_read(cache, C.cu_of([160, 3], DEV), 163)
        assert torch.equal(ko[:160], k[0].to(torch.bfloat16)) and (ko[160:] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_pages_past_2_31_elements(va, kind):
    """A pool whose last pages lie past 2^31 elements."""
    heads, dim, page = 8, 128, 64
    pages = 2 ** 31 // (page * heads * dim) + 40
    dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    pools = [torch.empty(pages, page, heads, dim, dtype=dt, device=DEV) for _ in range(2)]
    sc = [None if kind == "bf16" else torch.empty(pages, heads, page, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    n, ln = 150, 1000
    table = torch.arange(pages - 32, pages, dtype=torch.int32, device=DEV).reshape(2, 16)
    cache = va.PagedCache(pools[0], pools[1], table, torch.tensor([ln, ln], dtype=torch.int32, device=DEV), *sc)
    k, v = _q(2 * ln, heads, dim, 1), _q(2 * ln, heads, dim, 2)
    va.cache_write(cache, k, v, C.cu_of([ln, ln], DEV))
    ko, vo = va.cache_read(cache, C.cu_of([ln, ln], DEV), 2 * ln)
    if kind == "bf16":
        assert torch.equal(ko, k) and torch.equal(vo, v)
    for new in ([1, 1], [n, 2]):
        q = _q(sum(new), 16, dim, 9)
        out, lse = va.attention_fwd_paged(q, cache, C.cu_of(new, DEV), max_seqlen_q=max(new), causal=True)
        _ok(va)
        at = 0
        for b, m in enumerate(new):
            ref = C.attend(q[at:at + m], ko[b * ln:(b + 1) * ln].double(), vo[b * ln:(b + 1) * ln].double(),
                           float(torch.tensor(dim ** -0.5)), -1, 0)
            C.check_attend(out[at:at + m], lse[:, at:at + m], ref, dim, ln)
            at += m
