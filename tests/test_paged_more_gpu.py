"""More of the paged cache on a GPU: empty calls, stale codes, larger shapes
drawn at random, calls by way of the bounds-checking build, and the raw entry
points with a caller's workspace."""
import math
import os
import random
import subprocess
import sys

import pytest
import torch

from tests import paged_cases as C
from tests.test_paged_gpu import _attend, _ok, _q

pytestmark = pytest.mark.gpu

DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def va():
    from packed_variable_length_varlen_gb300 import varlen_attn
    return varlen_attn


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_nothing_to_do(va, kind):
    """No rows, no keys, no segments with rows."""
    cache, _, _ = C.make_cache([0, 0], 2, 64, 16, kind, DEV)
    cu = C.cu_of([0, 0], DEV)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    va.cache_write(cache, none, none, cu)
    k, v = va.cache_read(cache, cu, 0)
    assert k.shape == (0, 2, 64)
    out, lse = va.attention_fwd_paged(torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV), cache, cu)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    for rows in (3, 90):  # rows, but in no segment
        q = _q(rows, 4, 64)
        out = torch.full_like(q, 9.0)
        va.attention_fwd_paged(q, cache, cu, out=out)
        assert (out == 9.0).all()
        va.cache_write(cache, _q(rows, 2, 64), _q(rows, 2, 64), cu)
    for new in ([1, 2], [80, 3]):  # segments with rows and without keys
        out, lse = va.attention_fwd_paged(_q(sum(new), 4, 64), cache, C.cu_of(new, DEV))
        assert (out == 0).all() and (lse == -math.inf).all()
    _ok(va)


@pytest.mark.parametrize("n", [1, 9, 100])
def test_stale_codes_may_be_anything(va, n):
    """Codes that stand for NaN, and NaN scales, behind the sequence's end and before the window."""
    cache, k, v = C.make_cache([333], 2, 128, 64, "e4m3", DEV)
    left = 40
    first = 333 - n - left
    for t in (cache.k_pages, cache.v_pages):
        raw = t.view(torch.uint8)
        for pg in range(raw.shape[0]):
            pos = (cache.block_table[0] == pg).nonzero()
            base = int(pos[0]) * 64 if len(pos) else 10 ** 6
            for row in range(64):
                if not first <= base + row < 333:
                    raw[pg, row] = 0x7f if row % 2 else 0xff
    q = _q(n, 8, 128)
    out, lse = va.attention_fwd_paged(q, cache, C.cu_of([n], DEV), max_seqlen_q=n, causal=True, window=(left, -1))
    _ok(va)
    ref = C.attend(q, k[0][first:], v[0][first:], float(torch.tensor(128 ** -0.5)), left, 0)
    C.check_attend(out, lse, ref, 128, 333)


@pytest.mark.parametrize("seed", range(24))
def test_drawn_shapes(va, seed):
    """Shapes drawn over the whole range that the entry points allow, small enough for the plain form."""
    r = random.Random(seed)
    kind = r.choice(("bf16", "e4m3"))
    kv = r.choice((1, 2, 3, 8))
    group = r.choice((1, 2, 3, 5, 7, 8, 12, 16, 33))
    batch = r.choice((1, 2, 5, 40))
    most = r.choice((1, 4, 30, 250))
    new = [r.randint(0 if most > 1 else 1, most) for _ in range(batch)]
    lens = [r.randint(0, r.choice((20, 300, 2500))) for _ in range(batch)]
    _attend(va, new, lens, kv * group, kv, r.choice((64, 96, 128)), r.choice((16, 32, 64, 128, 256, 512, 1024)), kind,
            r.random() < 0.7, (r.choice((-1, -1, 0, 5, 100, 1000)), r.choice((-1, 0, 3, 64))),
            order=r.choice(("nhd", "hnd", "padded", "together")), hint=r.choice((0, max(new))), seed=seed,
            pad=r.choice((0, 8)), extra=r.randint(0, 3))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("heads,kv", [(2, 2), (8, 2), (21, 3)])
def test_both_kernels_in_one_call(va, kind, dim, heads, kv):
    """Tables wide enough for long sequences: each segment goes to the kernel that its own length calls for, and a
    unit that several CTAs share is joined for both."""
    wide = 64 * 160 * 128 // 1024  # columns of 1024 positions that two segments' tables need to be taken for long
    _attend(va, [130, 1, 0, 257, 5, 65, 33, 3, 1, 16], [700, 300, 40, 257, 128, 1000, 20, 0, 9000, 5], heads, kv, dim,
            1024, kind, True, columns=wide, extra=2)
    _attend(va, [1, 2, 300], [4000, 2500, 9000], heads, kv, dim, 1024, kind, True, (700, -1), columns=wide, pad=8)


@pytest.mark.parametrize("new", [[3, 1], [200, 5], [70]])
def test_raw_call_with_a_workspace_that_holds_anything(va, new):
    """The C entry point with a caller's workspace of just the size, full of NaN, between canaries; the same bits
    as a call with another one."""
    lens = [5000, 300][:len(new)]
    H, kv, D = 8, 2, 128
    cache, k, v = C.make_cache(lens, kv, D, 64, "e4m3", DEV)
    total = sum(new)
    q, cu = _q(total, H, D), C.cu_of(new, DEV)
    need = va.varlen_attn_fwd_paged_workspace_size(len(new), total, H, kv, D)
    got = []
    for fill in (0x00, 0xff, 0x7f):
        ws = torch.full((need + 512,), fill, dtype=torch.uint8, device=DEV)
        ws[need:] = 0xa5
        out = torch.empty(total, H, D, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(H, total, device=DEV)
        st = va.varlen_attn_fwd_paged(q, cu, len(new), total, H, 0, cache.struct, D ** -0.5, -1, 0, out, lse, ws, need)
        assert st == 0, va.varlen_attn_status_string(st)
        _ok(va)
        assert (ws[need:] == 0xa5).all()
        got.append((out, lse))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    # a table shared by every sequence (row stride 0), as the C struct allows
    if len(new) == 2:
        s = va.VarlenKvCache.from_buffer_copy(cache.struct)
        s.table_stride = 0
        both = torch.tensor([300, 300], dtype=torch.int32, device=DEV)
        s.seqlens = both.data_ptr()
        st = va.varlen_attn_fwd_paged(q, cu, 2, total, H, 0, s, D ** -0.5, -1, 0, out, lse, ws, need)
        assert st == 0
        _ok(va)
        ref = C.attend(q[new[0]:], k[0][:300], v[0][:300], float(torch.tensor(D ** -0.5)), -1, 0)
        C.check_attend(out[new[0]:], lse[:, new[0]:], ref, D, 300)


@pytest.mark.parametrize("n", [1, 9, 100])
@pytest.mark.parametrize("shift", [-121, -119, -60, 60, 118])
def test_value_scales_at_the_ends_of_their_range(va, n, shift):
    """Values near the least and the largest scale (2^-127 and beyond): the output is that of ordinary values times
    the same power of two, bit for bit where both are quantised alike, else within the roundings."""
    ln, dim, heads = 200, 64, 2
    k, v = _q(ln, heads, dim, 5), _q(ln, heads, dim, 6)
    q, cu = _q(n, 4, dim, 7), C.cu_of([n], DEV)
    got = []
    for e in (0, shift):
        cache, _, _ = C.make_cache([ln], heads, dim, 16, "e4m3", DEV)
        va.cache_write(cache, k, (v.double() * 2.0 ** e).to(torch.bfloat16), C.cu_of([ln], DEV))
        out, lse = va.attention_fwd_paged(q, cache, cu, max_seqlen_q=n, causal=True)
        _ok(va)
        kk, vv = va.cache_read(cache, C.cu_of([ln], DEV), ln)
        # held values from the codes: reading back rounds where bf16 is subnormal
        pos = torch.arange(ln, device=DEV)
        pg = cache.block_table[0].long()[pos // 16]
        held = cache.v_pages.view(torch.uint8)[pg, pos % 16].view(torch.float8_e4m3fn).double() * \
            cache.v_scale[pg, :, pos % 16].double()[..., None]
        o, _, A, S = C.attend(q, kk.double(), held, 0.125, -1, 0)
        assert torch.isfinite(out).all()
        # P to bf16 or f16, the score's sum and exp2, O to bf16 (2^-134: half of bf16's least step)
        tol = 2.0 ** -8 * (A + o.abs()) + 2.0 ** -14 * A + 2.0 ** -134
        d = (out.double() - o).abs()
        assert (d <= tol).all(), (e, float((d / tol).max()))
        got.append((out.double() * 2.0 ** -e, lse))
    assert torch.equal(got[0][1], got[1][1])
    if shift > -119:
        assert torch.equal(got[0][0], got[1][0])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 9, 100])
@pytest.mark.parametrize("shift", [-80, 80])
def test_queries_and_keys_of_opposite_sizes(va, kind, n, shift):
    """Queries times 2^shift and keys times 2^-shift: the same scores, the same bits."""
    ln, dim, heads = 200, 128, 2
    k, v = _q(ln, heads, dim, 5), _q(ln, heads, dim, 6)
    q, cu = _q(n, 4, dim, 7), C.cu_of([n], DEV)
    got = []
    for e in (0, shift):
        cache, _, _ = C.make_cache([ln], heads, dim, 32, kind, DEV)
        va.cache_write(cache, (k.double() * 2.0 ** -e).to(torch.bfloat16), v, C.cu_of([ln], DEV))
        got.append(va.attention_fwd_paged((q.double() * 2.0 ** e).to(torch.bfloat16), cache, cu, max_seqlen_q=n, causal=True))
        _ok(va)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_a_call_on_another_stream_waits_for_its_allocations(va):
    """What a call allocates on the current stream may still be in use there: the call on another stream comes after."""
    cache, k, v = C.make_cache([700], 2, 64, 16, "bf16", DEV)
    q, cu = _q(100, 4, 64), C.cu_of([100], DEV)
    want = va.attention_fwd_paged(q, cache, cu, causal=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        busy = torch.empty(100 * 4 * 64, dtype=torch.bfloat16, device=DEV)
        for _ in range(20):
            busy.fill_(1.0)
        del busy  # its memory goes to the next allocation while the fills are still to run
        out, lse = va.attention_fwd_paged(q, cache, cu, causal=True, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    with torch.cuda.stream(side):  # and the other way round, on the default stream
        out, lse = va.attention_fwd_paged(q, cache, cu, causal=True, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    handle = side.cuda_stream
    out, lse = va.attention_fwd_paged(q, cache, cu, causal=True, stream=handle)
    kk, vv = va.cache_read(cache, C.cu_of([700], DEV), 700, stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(kk, k[0].to(torch.bfloat16)) and torch.equal(vv, v[0].to(torch.bfloat16))
    _ok(va)


def test_bounds_checked_build():
    """The cases of the other file on the build whose kernels check every plain global access."""
    from packed_variable_length_varlen_gb300 import build
    lib = build.build(bounds=True)
    env = dict(os.environ, VARLEN_ATTN_LIB=lib)
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_paged_gpu.py", "-q", "-x", "-m", "gpu", "-k",
                        "write_then_read or few_rows or test_chunks or layouts or head_groups or long_cache or bad_pages",
                        "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]


def test_both_kernels_captured_and_repeated(va):
    """A call of four launches that overlap, captured with the write before it and replayed; and two of them at once."""
    new, lens = [1, 200, 3, 1], [5000, 900, 64, 2000]
    cache, _, _ = C.make_cache(lens, 2, 128, 64, "e4m3", DEV, columns=64 * 160 * 128 // 64 // 4)
    cu, total = C.cu_of(new, DEV), sum(new)
    k, v, q = _q(total, 2, 128, 1), _q(total, 2, 128, 2), _q(total, 8, 128, 3)

    def step():
        va.cache_write(cache, k, v, cu)
        return va.attention_fwd_paged(q, cache, cu, causal=True)

    want = step()
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        got = [step() for _ in range(3)]
    for _ in range(5):
        for o, l in got:
            o.zero_()
            l.zero_()
        g.replay()
        torch.cuda.synchronize()
        for o, l in got:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        res = [va.attention_fwd_paged(q, cache, cu, causal=True, stream=s) for s in streams]
        torch.cuda.synchronize()
        for o, l in res:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    _ok(va)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_both_kernels_follow_the_lengths(va, kind):
    """Lengths, rows and a page's place that change between the replays of a captured step of four launches."""
    new, lens = [1, 150, 2, 1], [3000, 2900, 900, 2000]
    cache, _, _ = C.make_cache(lens, 2, 64, 64, kind, DEV, columns=64 * 160 * 128 // 64 // 4, spare=8)
    cu, total = C.cu_of(new, DEV), sum(new)
    start = torch.tensor([200, 700, 60, 1500], dtype=torch.int32, device=DEV)
    grow = torch.tensor(new, dtype=torch.int32, device=DEV)
    k, v, q = _q(total, 2, 64, 1), _q(total, 2, 64, 2), _q(total, 4, 64, 3)
    first = cache.block_table.clone()
    pools = [t.clone() for t in (cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8))]
    scales = [None if t is None else t.clone() for t in (cache.k_scale, cache.v_scale)]

    def reset():
        cache.seqlens.copy_(start)
        cache.block_table.copy_(first)
        for t, old in zip((cache.k_pages, cache.v_pages), pools):
            t.view(torch.uint8).copy_(old)
        for t, old in zip((cache.k_scale, cache.v_scale), scales):
            if t is not None:
                t.copy_(old)

    def step():
        cache.seqlens.add_(grow)
        va.cache_write(cache, k, v, cu)
        return va.attention_fwd_paged(q, cache, cu, causal=True)

    def between(i):
        k.copy_(_q(total, 2, 64, 20 + i))
        if i == 2:  # the first sequence's first page and the last one's change places
            a, b = first[0, 0].clone(), first[3, 1].clone()
            cache.block_table[0, 0], cache.block_table[3, 1] = b, a

    want = []
    reset()
    for i in range(5):
        between(i)
        want.append([t.clone() for t in step()])
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        got = step()
    torch.cuda.synchronize()
    for _ in range(3):
        reset()
        for i in range(5):
            between(i)
            g.replay()
            for a, b in zip(got, want[i]):
                assert torch.equal(a, b)
    _ok(va)
