"""The bounds-checking build and a step's operators: it gives the normal build's bits and reports nothing; with every
extent emptied no store that it checks lands, and the call says so; and the operators' own tests run on it."""
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
    from tests import step_bounds_cases as B
    path = str(tmp_path / "step.pt")
    env = dict(os.environ, VARLEN_ATTN_LIB=build.build(bounds=True))
    r = subprocess.run([sys.executable, "-m", "tests.step_bounds_cases", path], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    got, ref = torch.load(path), B.run(va)
    assert got.pop("checked") and not ref.pop("checked")
    for name, g in got.items():
        assert g["status"] == 0 and ref[name]["status"] == 0 and ref[name]["slack"] == 0, name
        for a, b in zip(g["good"], ref[name]["good"]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
        assert g["slack"] == va.VARLEN_ERR_DEVICE_BOUNDS and g["kept"], name


def test_the_operators_tests_on_it():
    from packed_variable_length_varlen_gb300 import build
    env = dict(os.environ, VARLEN_ATTN_LIB=build.build(bounds=True))
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_step_gpu.py", "tests/test_tree_gpu.py", "-q", "-x", "-m", "gpu",
                        "-k", "not far_pages and not long_strides and not deep", "-p", "no:cacheprovider"], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
