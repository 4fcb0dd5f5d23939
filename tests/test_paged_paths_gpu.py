"""The paged attention's ways through its kernels, on a GPU: units of every
number of rows that several CTAs share, so that the joins take each of their
forms, against the plain 64-bit form."""
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


# A CTA takes at least two tiles of 64 keys: 300 keys are 3 parts of a unit, 1900 are 15, 2100 are 17, 9000 are 71.
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("tokens,group", [(1, 16), (2, 8), (5, 3), (17, 1), (6, 3), (3, 7), (4, 6), (3, 9), (4, 8), (1, 31)])
@pytest.mark.parametrize("keys", [300, 1900, 2100, 9000])
def test_units_of_few_rows_in_parts(va, kind, dim, tokens, group, keys):
    """One sequence, two key heads; up to 16 rows (bf16) or 32 (E4M3) a unit, in parts that warps join (up to 16) and
    that blocks do.  (bf16 units of more rows go to the kernel for many, whose join takes a row a warp.)"""
    _check(va, [tokens], [keys], 2 * group, 2, dim, 64, kind, tokens, sizes=[0.05, 1.0, 6.0], repeats=6)
