"""Loads that never come, in the trees' kernels, with contexts sized by the GPU's SMs: every CTA, the first one's too, has
two tiles at least, so that load 3 (V of CTA 0's second tile) is one that is waited for.

Tiles that a CTA gets: the kernel for few rows has at most three CTAs an SM and tiles of 64 keys, each one place in the
list, the one for many one CTA an SM and tiles of 128 keys, each four or five places; 9 tiles of 64 an SM over 2 key heads
are three for each CTA of the first and more than four of 128 for each of the second."""
import pytest
import torch

from tests import paged_cases as C
from tests.test_tree_gpu import _tree

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def va():
    from packed_variable_length_varlen_gb300 import varlen_attn
    return varlen_attn


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("which,new", [(3, [3]), (4, [100])])
@pytest.mark.parametrize("load", [0, 1, 3])
def test_a_load_of_the_first_cta(va, kind, which, new, load):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    keys = 64 * 9 * sms // 2
    assert va.varlen_attn_get_device_status() == 0
    cache, _, _ = C.make_cache([keys], 2, 64, 64, kind, DEV)
    q = torch.randn(sum(new), 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    masks = torch.full((sum(new), 4), -1, dtype=torch.int32, device=DEV)
    assert va.varlen_attn_debug_skip_load(which, load) == 0
    try:
        va.attention_fwd_paged_tree(q, cache, C.cu_of(new, DEV), masks, max_seqlen_q=max(new))
        st = va.varlen_attn_get_device_status()
    finally:
        va.varlen_attn_debug_skip_load(which, -1)
    assert st == va.VARLEN_ERR_TIMEOUT, va.varlen_attn_status_string(st)
    _tree(va, new, [keys], 4, 2, 64, 64, kind)
