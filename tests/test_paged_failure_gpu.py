"""Failure detection in the paged attention without a GPU fault: a producer
leaves one load out, the bounded waits for it run out, every role of the CTA
unwinds, the call reports a time-out, and the next call on the same context
and workspace is right."""
import time

import pytest
import torch

from tests import paged_cases as C

pytestmark = pytest.mark.gpu

DEV = "cuda"
FEW, MANY = 3, 4  # selectors of varlen_attn_debug_skip_load


@pytest.fixture(scope="module")
def va():
    from packed_variable_length_varlen_gb300 import varlen_attn
    return varlen_attn


# loads of CTA 0, K and V counted alike: 5000 keys are 79 tiles of 64 and 40 of 128, so CTA 0 has at least 2 tiles
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("which,new,columns", [(FEW, [1, 2], 1), (MANY, [200, 3], 1), (MANY, [150, 1], 1 << 14),
                                               (FEW, [150, 1], 1 << 14)])
@pytest.mark.parametrize("load", [0, 3])
def test_skipped_load_times_out_and_the_next_call_is_right(va, kind, which, new, columns, load):
    """1 << 14 columns of 64 positions: tables wide enough that both kernels run."""
    lens, heads, kv, dim = [5000, 900], 4, 2, 128
    cache, k, v = C.make_cache(lens, kv, dim, 64, kind, DEV, columns=columns)
    total, cu = sum(new), C.cu_of(new, DEV)
    q = torch.randn(total, heads, dim, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    out = torch.zeros_like(q)
    lse = torch.zeros(heads, total, device=DEV)
    need = va.varlen_attn_fwd_paged_workspace_size(len(new), total, heads, kv, dim)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)

    def call():
        va.attention_fwd_paged(q, cache, cu, max_seqlen_q=max(new), out=out, lse=lse, workspace=ws, causal=True)
        return va.varlen_attn_get_device_status()

    assert va.varlen_attn_get_device_status() == 0
    assert va.varlen_attn_debug_skip_load(which, load) == 0
    try:
        t0 = time.time()
        st = call()
        elapsed = time.time() - t0
    finally:
        va.varlen_attn_debug_skip_load(which, -1)
    assert st == va.VARLEN_ERR_TIMEOUT, va.varlen_attn_status_string(st)
    assert 1.5 < elapsed < 30
    assert call() == 0
    at = 0
    for b, n in enumerate(new):
        ref = C.attend(q[at:at + n], k[b], v[b], float(torch.tensor(dim ** -0.5)), -1, 0)
        C.check_attend(out[at:at + n], lse[:, at:at + n], ref, dim, lens[b])
        at += n
