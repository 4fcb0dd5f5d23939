"""Writes into the paged cache that have no place, on a GPU: they leave what is
there as it was, and the status says so."""
import pytest
import torch

from tests import paged_cases as C

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def va():
    from packed_variable_length_varlen_gb300 import varlen_attn
    return varlen_attn


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("past", [1, 5, 16, 64, 2 ** 31 - 1 - 192])
def test_rows_past_the_table_are_dropped(va, kind, page, past):
    """A length that has grown past what its table row can name: the rows that have no page are dropped and reported,
    the ones before them go to their own places, and no older row is written over."""
    cap, heads, dim, n = 192, 2, 64, 8
    cache, k, v = C.make_cache([cap, 40], heads, dim, page, kind, DEV, columns=cap // page)
    cache.seqlens[0] = cap + past
    g = torch.Generator().manual_seed(1)
    kn, vn = (torch.randn(n + 3, heads, dim, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    va.cache_write(cache, kn, vn, C.cu_of([n, 3], DEV))
    assert va.varlen_attn_get_device_status() == va.VARLEN_ERR_DEVICE_BOUNDS
    for held, new in ((k, kn), (v, vn)):
        if kind == "e4m3":
            codes, s = C.quantise(new)
            new = codes.double() * s.double()[..., None]
        stay = max(n - past, 0)
        held[0][cap + past - n:] = new[:stay].double() if stay else held[0][cap + past - n:]
        held[1][37:] = new[n:].double()
    cache.seqlens[0] = cap
    ko, vo = va.cache_read(cache, C.cu_of([cap, 40], DEV), cap + 40)
    assert va.varlen_attn_get_device_status() == 0
    for got, held in ((ko, k), (vo, v)):
        assert torch.equal(got, torch.cat(held).to(torch.bfloat16))
