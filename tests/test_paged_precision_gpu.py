"""What the paged attention keeps of small weights, on a GPU: a first key that
takes nearly all of a row's weight and whose value is zero, so that the output
is made of many keys far below it, beside values and scales of other sizes."""
import pytest
import torch

from tests import paged_cases as C

pytestmark = pytest.mark.gpu

DEV = "cuda"
DIM, KEYS = 128, 6000


@pytest.fixture(scope="module")
def va():
    from packed_variable_length_varlen_gb300 import varlen_attn
    return varlen_attn


def _call(va, kind, tokens, heads, gap, value, seed=0):
    """Key 0 scores `gap` (as a power of two) above all others; value(k, v, c) changes the keys and values
    [KEYS, 1, DIM].  The check is that of the other tests: weights to 2^-8 of themselves, whatever their size."""
    g = torch.Generator().manual_seed(seed)
    c = 8.0 * DIM ** -0.5 / 0.6931471805599453  # scores in powers of two per unit of a key's first element
    k = torch.zeros(KEYS, 1, DIM, device=DEV)
    k[0, 0, 0] = gap / c
    v = (torch.rand(KEYS, 1, DIM, generator=g) * 0.04 + 0.06).to(DEV)  # largest 0.1: a scale of 2^-12
    v[0] = 0
    value(k, v, c)

    def fill(x, b, i):
        return (k if i == 0 else v).to(torch.bfloat16)

    cache, kk, vv = C.make_cache([KEYS], 1, DIM, 64, kind, DEV, fill=fill)
    q = torch.zeros(tokens, heads, DIM, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 8.0
    out, lse = va.attention_fwd_paged(q, cache, C.cu_of([tokens], DEV), max_seqlen_q=tokens)
    assert va.varlen_attn_get_device_status() == 0
    ref = C.attend(q, kk[0], vv[0], float(torch.tensor(DIM ** -0.5, dtype=torch.float32)), -1, -1)
    C.check_attend(out, lse, ref, DIM, KEYS)


ROWS = [(1, 1), (1, 8), (2, 12), (40, 4)]  # tokens and heads: one to three row tiles, and the kernel for many rows
GAPS = [0.0, 9.5, 14.3, 17.7, 20.4]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens,heads", ROWS)
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("every", [1, 16, 500, 6000])
def test_zero_vectors_say_nothing_of_the_sizes(va, kind, tokens, heads, gap, every):
    """A vector of zeros has a scale of one, 2^12 of its neighbours': it takes nothing from their weights."""
    def value(k, v, c):
        v[::every] = 0

    _call(va, kind, tokens, heads, gap, value)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens,heads", ROWS)
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("size", [4, 7, 8, 9, 11, 12, 13, 40])
def test_large_values_of_small_weight(va, kind, tokens, heads, gap, size):
    """A few values 2^size times the others', whose own weight is 2^-30 of theirs."""
    def value(k, v, c):
        v[5::1500] *= 2.0 ** size
        k[5::1500, 0, 0] = -30 / c

    _call(va, kind, tokens, heads, gap, value)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens,heads", ROWS)
@pytest.mark.parametrize("gap", GAPS)
def test_values_that_grow(va, kind, tokens, heads, gap):
    """Sizes that rise by 2^30 along the cache in small steps, so that the largest scale moves again and again."""
    def value(k, v, c):
        v *= torch.exp2(torch.linspace(-15, 15, KEYS, device=DEV))[:, None, None]

    _call(va, kind, tokens, heads, gap, value)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 9, 100])
@pytest.mark.parametrize("shift", [-122, -116, -104, 104, 116, 122])
def test_queries_and_keys_at_opposite_ends_of_the_range(va, kind, n, shift):
    """Queries times 2^shift and keys times 2^-shift: the same scores.  Up to 2^104 the same bits as well, as every
    number keeps its own: the least are near 2^-20, and bf16 is normal down to 2^-126.  Beyond, the smaller side
    holds subnormal numbers, which are not those of the unshifted call any more: the check is the plain form's on the
    numbers that there are."""
    ln, dim, heads = 200, 128, 2
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(ln, heads, dim, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    q, cu = torch.randn(n, 4, dim, generator=g).to(torch.bfloat16).to(DEV), C.cu_of([n], DEV)
    got = []
    for e in (0, shift):
        cache, _, _ = C.make_cache([ln], heads, dim, 32, kind, DEV)
        ke, qe = (k.double() * 2.0 ** -e).to(torch.bfloat16), (q.double() * 2.0 ** e).to(torch.bfloat16)
        va.cache_write(cache, ke, v, C.cu_of([ln], DEV))
        got.append(va.attention_fwd_paged(qe, cache, cu, max_seqlen_q=n, causal=True))
        assert va.varlen_attn_get_device_status() == 0
        kh, vh = ke.double(), v.double()
        if kind == "e4m3":
            (kc, ks), (vc, vs) = C.quantise(ke), C.quantise(v)
            kh, vh = kc.double() * ks.double()[..., None], vc.double() * vs.double()[..., None]
        ref = C.attend(qe, kh, vh, float(torch.tensor(dim ** -0.5, dtype=torch.float32)), -1, 0)
        C.check_attend(got[-1][0], got[-1][1], ref, dim, ln)
    if abs(shift) <= 104:
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 8), (2, 8), (5, 3)])  # at most 16 rows
def test_few_rows_add_nothing_to_the_outputs_own_rounding(va, kind, tokens, heads):
    """Units of few rows: half a step of bf16 for the output (2^-8 of it), and of the sum of its terms' sizes 2^-16 for
    weights in two bf16 parts (bf16 cache; each part's rounding at most 2^-8 of what it rounds) or 2^-11 for weights in
    f16 (E4M3), beside the scores' errors (fp32 sums of DIM products, exp2).  All keys but the first have one weight, at
    sixteen places between two powers of two, so that its rounding does not average out."""
    c = 8.0 * DIM ** -0.5 / 0.6931471805599453
    g = torch.Generator().manual_seed(3)
    v = (torch.rand(300, 1, DIM, generator=g) + 0.5).to(torch.bfloat16).to(DEV)
    q = torch.zeros(tokens, heads, DIM, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 8.0
    for i in range(16):
        k = torch.zeros(300, 1, DIM, device=DEV)
        k[0, 0, 0] = (1 + i / 16) / c
        cache, kk, vv = C.make_cache([300], 1, DIM, 64, kind, DEV, fill=lambda x, b, n: k.to(torch.bfloat16) if n == 0 else v)
        out, _ = va.attention_fwd_paged(q, cache, C.cu_of([tokens], DEV), max_seqlen_q=tokens)
        assert va.varlen_attn_get_device_status() == 0
        o, _, A, S = C.attend(q, kk[0], vv[0], float(torch.tensor(DIM ** -0.5, dtype=torch.float32)), -1, -1)
        e = (DIM + 8) * 2.0 ** -24 * S.T[..., None] + 2.0 ** -21 + (300 / 16 + 64) * 2.0 ** -24
        tol = 2.0 ** -8 * o.abs() + (2.0 ** (-16 if kind == "bf16" else -11) + 2 * e) * A
        d = (out.double() - o).abs()
        assert (d <= tol).all(), (i, float((d / tol).max()))
