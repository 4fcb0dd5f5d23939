"""Rules that the sources of a step's kernels keep, read on the CPU (see test_paged_sources for why)."""
import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parents[1] / "packed_variable_length_varlen_gb300" / "csrc"
KERNELS = {"varlen_rotary.cu": {"varlen_rotary_kernel"},
           "varlen_plan.cu": {"varlen_plan_kernel", "varlen_plan_rows_kernel", "varlen_plan_trees_kernel", "varlen_trim_kernel",
                              "varlen_move_kernel"}}


def _source(name):
    return re.sub(r"//.*", "", (CSRC / name).read_text())


def _kernels(name):
    text = _source(name)
    for m in re.finditer(r"__global__ void[^{;]*?(varlen_\w+_kernel)\([^{;]*\{", text):
        body = text[m.end():]
        yield m.group(1), body[:body.index("\n}\n")]


def test_overlapped_kernels_wait_before_they_touch_memory():
    for name, want in KERNELS.items():
        seen = set()
        for kernel, body in _kernels(name):
            waits = re.findall(r"dependency_wait\(\);", body)
            at = re.search(r"^  dependency_wait\(\);", body, re.M)
            assert len(waits) == 1 and at, kernel
            assert not re.search(r"\bp\.|->|return", body[:at.start()]), kernel
            seen.add(kernel)
        assert seen == want
        launches = re.findall(r"<<<", _source(name))
        assert not launches  # all are launched to overlap


def test_overlapped_kernels_read_with_ordinary_loads():
    for name in list(KERNELS) + ["varlen_step.h", "varlen_e4m3.cuh"]:
        assert not re.search(r"__ldg|__ldlu|ld\.global\.nc|__restrict__", _source(name)), name


def test_pieces_that_are_read_where_they_lie_are_given_back():
    """The tree form of the kernel for many rows leaves a piece in the ring while it works on it: every way to the next
    piece gives it back first."""
    text = _source("varlen_paged_chunk.cu")
    roles = [r for r in re.split(r"\n    while \(ok", text)[1:] if r.startswith(" && (TREE ? pieces.wait")]
    assert len(roles) == 2  # softmax, conversion
    softmax, convert = roles
    for m in re.finditer(r"\bcontinue;", softmax[:softmax.index("\n    }\n")]):
        assert "pieces.done(sh);" in softmax[max(0, m.start() - 60):m.start()]
    assert "if (TREE) pieces.done(sh);\n      g += tiles;" in softmax
    assert "if (TREE && ok) pieces.done(sh);" in convert
