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
