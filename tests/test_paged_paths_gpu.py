"""The paged attention's ways through its kernels, on a GPU, against the plain
64-bit form: units of every number of rows that several CTAs share, so that the
joins take each of their forms; hints that choose the kernel for few rows at
every group size; and each call with tables that make one kernel take all of
it and with tables wide enough that both run."""
import random

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


def _rows(total, heads, dim, seed, sizes=None):
    """Random bf16 queries; `sizes` multiplies (token, head) rows, so that their maxima differ strongly."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(total, heads, dim, generator=g)
    if sizes is not None:
        q *= torch.tensor(sizes)[torch.randint(0, len(sizes), (total, heads), generator=g)][..., None]
    return q.to(torch.bfloat16).to(DEV)


def _check(va, new, lens, heads, kv, dim, page, kind, hint, columns=1, sizes=None, repeats=1, seed=0, window=(-1, -1)):
    """The call against the plain form, and its repeats bit for bit."""
    def fill(x, b, i):  # key sizes that grow, so that the parts of a unit have different maxima
        ramp = torch.linspace(0.2, 2.0, max(x.shape[0], 1), device=x.device)[:, None, None]
        return x if i == 1 else (x.float() * ramp).to(torch.bfloat16)

    cache, k, v = C.make_cache(lens, kv, dim, page, kind, DEV, seed=seed, fill=fill, columns=columns)
    q, cu = _rows(sum(new), heads, dim, seed + 1, sizes), C.cu_of(new, DEV)
    out, lse = va.attention_fwd_paged(q, cache, cu, max_seqlen_q=hint, causal=True, window=window)
    _ok(va)
    at = 0
    for b, n in enumerate(new):
        ref = C.attend(q[at:at + n], k[b], v[b], float(torch.tensor(dim ** -0.5, dtype=torch.float32)), window[0], 0)
        C.check_attend(out[at:at + n], lse[:, at:at + n], ref, dim, lens[b])
        at += n
    for _ in range(repeats - 1):
        o, l = va.attention_fwd_paged(q, cache, cu, max_seqlen_q=hint, causal=True, window=window)
        assert torch.equal(o, out) and torch.equal(l, lse)
    _ok(va)


def _wide(batch, kv, page):
    """Table columns with which a call of several segments is taken for long whatever its lengths are: 256 tiles of
    128 keys for each of 160 SMs."""
    return -(-256 * 160 * 128 // (batch * kv * page))


# A CTA takes at least two tiles of 64 keys: 300 keys are 3 parts of a unit, 1900 are 15, 2100 are 17, 9000 are 71.
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("tokens,group", [(1, 16), (2, 8), (5, 3), (17, 1), (6, 3), (3, 7), (4, 6), (3, 9), (4, 8), (1, 31)])
@pytest.mark.parametrize("keys", [300, 1900, 2100, 9000])
def test_units_of_few_rows_in_parts(va, kind, dim, tokens, group, keys):
    """One sequence, two key heads; up to 16 rows a unit, in parts that warps join (up to 16) and that blocks do, and
    up to 32, which the kernel for many rows takes (its join takes a row a warp)."""
    _check(va, [tokens], [keys], 2 * group, 2, dim, 64, kind, tokens, sizes=[0.05, 1.0, 6.0], repeats=6)


LENS = [5, 7, 0, 200, 64, 16, 700, 3, 129, 65, 2100]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("group,kv,page", [(1, 2, 16), (3, 2, 128), (4, 1, 64), (7, 2, 32), (8, 1, 16), (16, 1, 256)])
@pytest.mark.parametrize("window", [(-1, -1), (37, -1)])
def test_the_kernel_for_few_rows_at_every_group(va, kind, dim, group, kv, page, window):
    """Segments of up to 16 rows with the hint that says so: no other kernel takes part."""
    most = 16 // group
    r = random.Random(group)
    new = [most, 0, 1] + [r.randint(0, most) for _ in LENS[3:]]
    _check(va, new, LENS, group * kv, kv, dim, page, kind, most, window=window)


NEW = [130, 1, 0, 257, 4, 65, 33, 2, 1, 1, 3]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("group,kv,page", [(1, 2, 16), (4, 2, 64), (7, 1, 32), (3, 1, 1024), (8, 2, 128), (20, 1, 64)])
@pytest.mark.parametrize("hint", [0, 257])
@pytest.mark.parametrize("wide", [False, True])
def test_chunks_beside_tokens_both_ways(va, kind, dim, group, kv, page, hint, wide):
    _check(va, NEW, LENS, group * kv, kv, dim, page, kind, hint, columns=_wide(len(NEW), kv, page) if wide else 1,
           repeats=2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hint", [0, 1, 2, 1000000])
@pytest.mark.parametrize("wide", [False, True])
def test_hints_both_ways(va, kind, hint, wide):
    _check(va, [1, 200, 7], [300, 800, 64], 4, 2, 128, 64, kind, hint, columns=_wide(3, 2, 64) if wide else 1)


@pytest.mark.parametrize("seed", range(16))
@pytest.mark.parametrize("wide", [False, True])
def test_drawn_shapes_both_ways(va, seed, wide):
    r = random.Random(100 + seed)
    kv, group, batch = r.choice((1, 2, 3, 8)), r.choice((1, 2, 3, 5, 7, 8, 12, 16, 33)), r.choice((2, 5, 40))
    page, most = r.choice((16, 32, 64, 128, 256, 512, 1024)), r.choice((4, 30, 250))
    new = [r.choice((1, 1, r.randint(0, most))) for _ in range(batch)]
    lens = [r.randint(0, r.choice((20, 300, 2500))) for _ in range(batch)]
    _check(va, new, lens, kv * group, kv, r.choice((64, 96, 128)), page, r.choice(("bf16", "e4m3")), r.choice((0, max(new))),
           columns=_wide(batch, kv, page) if wide else 1, window=(r.choice((-1, -1, 0, 5, 100, 1000)), -1), seed=seed)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_both_kernels_on_several_streams(va, kind):
    """Calls of both kernels, several at once, each with its own workspace: the bits of a call alone."""
    new, lens = [40, 1, 3], [5000, 3000, 700]
    cache, _, _ = C.make_cache(lens, 2, 128, 64, kind, DEV, columns=_wide(3, 2, 64))
    cu = C.cu_of(new, DEV)
    qs = [_rows(sum(new), 8, 128, s) for s in (1, 2, 3)]
    alone = [va.attention_fwd_paged(q, cache, cu, causal=True) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(8):
        got = [va.attention_fwd_paged(q, cache, cu, causal=True, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for (o, l), (o1, l1) in zip(alone, got):
            assert torch.equal(o, o1) and torch.equal(l, l1)
    _ok(va)
