"""The bounds-checking build and the paged attention: calls whose units lie in
parts give the normal build's bits and report nothing; with every extent
emptied no store lands, in the outputs or in the workspace, and the call says
so; and the calls that take each way through the kernels, both in one call
among them, run on it."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_plain_access_is_checked(tmp_path):
    from packed_variable_length_varlen_gb300 import build
    from packed_variable_length_varlen_gb300 import varlen_attn as va
    from tests import paged_bounds_cases as B
    path = str(tmp_path / "paged.pt")
    env = dict(os.environ, VARLEN_ATTN_LIB=build.build(bounds=True))
    r = subprocess.run([sys.executable, "-m", "tests.paged_bounds_cases", path], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    got, ref = torch.load(path), B.run(va)
    assert got.pop("checked") and not ref.pop("checked")
    for name, g in got.items():
        want = ref[name]["good"]
        assert g["good"]["status"] == 0 and want["status"] == 0 and g["good"]["workspace_used"], name
        assert torch.equal(g["good"]["out"], want["out"]) and torch.equal(g["good"]["lse"], want["lse"]), name
        assert g["status"] == va.VARLEN_ERR_DEVICE_BOUNDS, name
        assert g["out_kept"] and g["lse_kept"] and g["workspace_kept"], (name, g)
        assert ref[name]["status"] == 0  # the normal build carries no checks


def test_every_way_through_the_kernels():
    """The cases of the other files in which units lie in parts, hints choose a kernel, or both kernels run."""
    from packed_variable_length_varlen_gb300 import build
    env = dict(os.environ, VARLEN_ATTN_LIB=build.build(bounds=True))
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_paged_paths_gpu.py", "tests/test_paged_more_gpu.py",
                        "-q", "-x", "-m", "gpu", "-k", "in_parts or every_group or both_ways or both_kernels or drawn",
                        "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
