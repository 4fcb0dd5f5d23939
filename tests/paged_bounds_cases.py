"""Calls of the paged attention with every extent emptied, for the
bounds-checking build (run by tests/test_paged_bounds_gpu.py with
VARLEN_ATTN_LIB pointing at that build): no plain store lands anywhere.

    python -m tests.paged_bounds_cases OUT.pt
"""
import sys

import torch

from tests import paged_cases as C

DEV = "cuda"
# new rows, table columns: the kernel for few rows, the one for many, both (wide tables), all with units in parts
CALLS = {"few": ([1, 2], 1), "many": ([200, 3], 1), "both": ([150, 1], 1 << 14)}


def run(va):
    res = {"checked": va.varlen_attn_bounds_checked()}
    for kind in ("bf16", "e4m3"):
        for name, (new, columns) in CALLS.items():
            heads, kv, dim = 4, 2, 128
            cache, _, _ = C.make_cache([5000, 900], kv, dim, 64, kind, DEV, columns=columns)
            total, cu = sum(new), C.cu_of(new, DEV)
            q = torch.randn(total, heads, dim, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
            need = va.varlen_attn_fwd_paged_workspace_size(len(new), total, heads, kv, dim)

            def call():
                out, lse = torch.full_like(q, 7.0), torch.full((heads, total), 7.0, device=DEV)
                ws = torch.full((need,), 0xa5, dtype=torch.uint8, device=DEV)
                va.attention_fwd_paged(q, cache, cu, max_seqlen_q=max(new), out=out, lse=lse, workspace=ws, causal=True)
                return va.varlen_attn_get_device_status(), out, lse, ws

            st, out, lse, ws = call()
            good = {"status": st, "out": out.cpu(), "lse": lse.cpu(), "workspace_used": bool((ws != 0xa5).any())}
            va.varlen_attn_debug_set_span_slack(1 << 60)
            try:
                st, out, lse, ws = call()
            finally:
                va.varlen_attn_debug_set_span_slack(0)
            res[kind + "/" + name] = {"good": good, "status": st, "out_kept": bool((out == 7.0).all()),
                                      "lse_kept": bool((lse == 7.0).all()),
                                      "workspace_kept": bool((ws == 0xa5).all())}
    return res


if __name__ == "__main__":
    from packed_variable_length_varlen_gb300 import varlen_attn
    torch.save(run(varlen_attn), sys.argv[1])
