"""Rules that the sources of the paged attention's kernels keep, read on the
CPU: what they guard against (data read before it is complete, a warp that
parts at a wait) shows on a GPU as a wrong result or a hang once in a long
while, if at all."""
import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parents[1] / "packed_variable_length_varlen_gb300" / "csrc"
KERNEL_FILES = ("varlen_paged.cu", "varlen_paged_few.cu", "varlen_paged_chunk.cu")


def _source(name):
    """The file's text without comments (role headings, `// ------ name`, are kept)."""
    text = (CSRC / name).read_text()
    return re.sub(r"//(?! ?-{4,}).*", "", text)


def _kernels():
    """(name, body) of every kernel that is launched to overlap with the one before it."""
    for f in KERNEL_FILES:
        text = _source(f)
        for m in re.finditer(r"__global__ void[^{;]*?(varlen_paged_\w+_kernel)\([^{;]*\{", text):
            body = text[m.end():]
            yield m.group(1), body[:body.index("\n}\n")]


def test_overlapped_kernels_wait_before_they_touch_memory():
    """A grid that may start while the one before it on the stream still runs sees nothing of what that one (or any
    before it) wrote until its own wait returns: each kernel waits once, whatever its arguments, before its first read."""
    seen = []
    for name, body in _kernels():
        waits = [m.start() for m in re.finditer(r"dependency_wait\(\)", body)]
        plain = [m.start() for m in re.finditer(r"^  dependency_wait\(\);", body, re.M)]
        assert len(plain) == 1 and plain[0] + 2 == waits[-1], name
        before = body[:plain[0]]
        assert not re.search(r"__ldg|paged_start|paged_note|p\.(cu_q|pages|q\b|out|lse)|parts\.|tma_load", before), name
        seen.append(name)
    assert sorted(seen) == ["varlen_paged_chunk_kernel", "varlen_paged_few_kernel", "varlen_paged_join_kernel",
                            "varlen_paged_join_rows_kernel"]


def test_overlapped_kernels_read_with_ordinary_loads():
    """The non-coherent path (__ldg, ld.global.nc) is for data that nobody writes while the kernel lives; a kernel that
    started early lives while the ones before it still write the lengths, the table and the queries."""
    for f in KERNEL_FILES + ("varlen_paged_walk.cuh", "varlen_paged.h"):
        assert not re.search(r"__ldg|__ldlu|ld\.global\.nc|__restrict__", _source(f)), f


def test_a_warp_parts_its_rows_in_the_join():
    """A warp joins row after row through the same weights in shared memory: it comes together after the last read of
    one row's (the divergent store of the row's LSE is no meeting point) and before the first write of the next one's."""
    text = _source("varlen_paged.cu")
    body = text[text.index("void join_by_warp("):]
    body = body[:body.index("\n}\n")]
    assert body.rstrip().endswith("__syncwarp();")
    assert body.index("weight[2 * k] = ex2") < body.index("__syncwarp();") < body.index("o[i] = fmaf(")


def test_a_kernel_that_returns_early_leaves_the_join_nothing():
    """The workspace holds anything on entry and the join follows what it finds there: a CTA that gives up before its
    producer cleared its entries clears them itself (after the wait)."""
    for name, body in _kernels():
        for m in re.finditer(r"^ {2,}return;", body, re.M):
            assert body[:m.start()].rstrip().endswith("paged_refuse(p, parts);"), name
    walk = _source("varlen_paged_walk.cuh")
    body = walk[walk.index("void paged_refuse("):]
    body = body[:body.index("\n}\n")]
    assert body.index("dependency_wait();") < body.index("clear_join(p, parts);") < body.index("record_error")


def test_a_wait_that_can_give_up_has_one_outcome_for_a_warp():
    """Every wait whose failure makes a role leave is voted on by the whole warp (mbar_wait_warp, warp_wait), but for
    the product issuer's, which is one thread: lanes that leave one by one would leave the others at the warp's next
    __syncwarp."""
    few = _source("varlen_paged_few.cu")
    assert not re.findall(r"!\s*mbar_wait\(", few)
    roles = re.split(r"// -{4,} (.*)", _source("varlen_paged_chunk.cu"))
    names = [r.strip() for r in roles[1::2]]
    assert names == ["producer", "MMA issuer", "clearing (bf16)", "softmax", "codes to bf16"]
    for name, body in zip(names, roles[2::2]):
        alone, voted = re.findall(r"!\s*mbar_wait\(", body), re.findall(r"!\s*mbar_wait_warp\(", body)
        reader = re.findall(r"PieceReader<(\w+)>", body)
        if name == "MMA issuer":
            assert alone and not voted and reader == ["false"]
        else:
            assert voted and not alone and reader in ([], ["true"]), name
