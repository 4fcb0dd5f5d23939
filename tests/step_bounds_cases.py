"""A step's operators with every extent emptied, for the bounds-checking build (run by tests/test_step_bounds_gpu.py with
VARLEN_ATTN_LIB pointing at that build): no plain store to what the checks cover lands anywhere.

    python -m tests.step_bounds_cases OUT.pt
"""
import sys

import torch

from tests import paged_cases as C
from tests import step_cases as S

DEV = "cuda"


def run(va):
    res = {"checked": va.varlen_attn_bounds_checked()}

    def both(name, make):
        """make() -> (call, what it may write)"""
        call, outs = make()
        call()
        st = va.varlen_attn_get_device_status()
        good = [t.cpu().clone() for t in outs]
        call, outs = make()
        before = [t.clone() for t in outs]
        va.varlen_attn_debug_set_span_slack(1 << 60)
        try:
            call()
            slack = va.varlen_attn_get_device_status()
        finally:
            va.varlen_attn_debug_set_span_slack(0)
        kept = all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, before))
        res[name] = {"good": good, "status": st, "slack": slack, "kept": kept}

    def rows(n, h, seed, dim=128):
        return torch.randn(n, h, dim, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)

    def ints(v, dt=torch.int32):
        return torch.tensor(v, dtype=dt, device=DEV)

    for rot in (128, 24):
        rope = va.Rotary(va.rotary_frequencies(rot)[0], device=DEV)

        def rotary():
            q, k = rows(9, 5, 1), rows(9, 2, 2)
            qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
            return (lambda: va.rotary(q, k, rope, ints(list(range(9))), None, qo, ko)), [qo, ko]

        both("rotary/%d" % rot, rotary)
        for kind in ("bf16", "e4m3"):
            def write():
                c, _, _ = C.make_cache([40], 3, 128, 16, kind, DEV)
                q, k, v = rows(9, 5, 1), rows(9, 3, 2), rows(9, 3, 3)
                qo = torch.full_like(q, 7.0)
                out = [qo, c.k_pages, c.v_pages] + [s for s in (c.k_scale, c.v_scale) if s is not None]
                return (lambda: va.rotary_cache_write(c, q, k, v, rope, ints(list(range(9))), ints(list(range(20, 29)), torch.int64), qo)), out

            both("write/%s/%d" % (kind, rot), write)
    for kind in ("bf16", "e4m3"):
        def move():
            c, _, _ = C.make_cache([40, 30], 3, 128, 16, kind, DEV)
            out = [c.k_pages, c.v_pages] + [s for s in (c.k_scale, c.v_scale) if s is not None]
            return (lambda: va.cache_move(c, C.cu_of([20, 9], DEV), ints([[3, 9, 19], [1, 2, 4]]), ints([3, 3]))), out

        both("move/" + kind, move)
        for name, (new, columns) in {"few": ([3, 2], 1), "many": ([90, 3], 1), "both": ([70, 1], 1 << 14)}.items():
            def tree():
                heads, kv, dim = 4, 2, 128
                c, _, _ = C.make_cache([5000, 900], kv, dim, 64, kind, DEV, columns=columns)
                q, g = rows(sum(new), heads, 4), torch.Generator().manual_seed(1)
                words = -(-max(new) // 32)
                masks = torch.cat([S.pack(S.ancestors(S.random_tree(n, g)), words) for n in new]).to(DEV)
                out, lse = torch.full_like(q, 7.0), torch.full((heads, sum(new)), 7.0, device=DEV)
                ws = torch.full((va.varlen_attn_fwd_paged_workspace_size(2, sum(new), heads, kv, dim),), 0xa5, dtype=torch.uint8, device=DEV)
                pos = ints([4990] * new[0] + [890] * new[1])
                return (lambda: va.attention_fwd_paged_tree(q, c, C.cu_of(new, DEV), masks, max_seqlen_q=max(new), window_left=700, positions=pos,
                                                            out=out, lse=lse, workspace=ws)), [out, lse]

            both("tree/%s/%s" % (kind, name), tree)
    for new in ([5, 3], [3000, 40]):
        for trees in (False, True):
            def plan():
                pool = va.PagePool(torch.zeros(2, 200, dtype=torch.int32, device=DEV), ints([5, 0]), torch.arange(300, dtype=torch.int32, device=DEV), ints([300]), 16)
                p = va.StepPlan(2, sum(new) + 3, DEV, mask_words=128 if trees else 0)
                out = [t.fill_(7) for t in (p.slots, p.positions, p.masks) if t is not None]
                up = sum([S.random_tree(n, torch.Generator().manual_seed(n)) for n in new], []) + [0] * 3
                return (lambda: va.cache_plan(pool, p, ints(new), ints(up) if trees else None)), out

            both("plan/%d/%d" % (new[0], trees), plan)

    def trim():
        free = torch.full((40,), 7, dtype=torch.int32, device=DEV)
        pool = va.PagePool(torch.arange(20, dtype=torch.int32, device=DEV).reshape(2, 10), ints([150, 100]), free, ints([1]), 16)
        return (lambda: va.cache_trim(pool, ints([3, 50]))), [free]

    both("trim", trim)
    return res


if __name__ == "__main__":
    from packed_variable_length_varlen_gb300 import varlen_attn
    torch.save(run(varlen_attn), sys.argv[1])
