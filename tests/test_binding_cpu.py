"""CPU checks of what the binding needs to load, and of its answers to missing arguments. No
GPU is touched: every call here fails a check, or asks only for sizes."""
import os
import subprocess
import sys

import pytest

from combine_ep_get_03_amd import _binding
from combine_ep_get_03_amd import build as hip_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT_THE_TENSOR_CHECK = """
import torch
import combine_ep_get_03_amd as ep
from combine_ep_get_03_amd import _binding
_binding.TENSOR_PTR_PATH = _binding.TENSOR_PTR_PATH + ".absent"
assert ep.ep_layout_workspace_bytes(256, 16, 4, 2) > 0
assert ep.ep_rmsnorm_grad_workspace_bytes(4, 256) > 0
assert ep.ep_status_string(0)
x = torch.zeros((4, 256), dtype=torch.bfloat16)
try:
    ep.ep_dispatch_permute(x, None, torch.zeros((4, 2), dtype=torch.int32), perm_x=x)
except ValueError as e:
    assert "device tensor" in str(e), e
else:
    raise AssertionError("host tensors taken")
for call in (lambda: ep.ep_rmsnorm(x, x[0], y=x),
             lambda: ep.ep_combine_unpermute(x, None, torch.zeros((4, 2), dtype=torch.int32), out=x)):
    try:
        call()
    except RuntimeError as e:
        assert "_tensor_ptr.so.absent is not built" in str(e), e
    else:
        raise AssertionError("the call went on without its check")
print("done")
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    if not (os.path.exists(_binding.LIB_PATH) and os.path.exists(_binding.TENSOR_PTR_PATH)):
        import __graft_entry__

        __graft_entry__.build()


def test_only_the_calls_that_use_the_tensor_check_need_it():
    """libep.so alone serves the layout, dispatch and combine calls and the size queries; the
    norm and expert-row calls say what is missing."""
    r = subprocess.run([sys.executable, "-c", WITHOUT_THE_TENSOR_CHECK], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr


def test_building_the_library_builds_the_tensor_check(monkeypatch, tmp_path):
    """One call makes all that the binding loads; a library elsewhere is built alone. The
    compilers are a stand-in that creates its output."""
    fake = tmp_path / "cc"
    fake.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\n: > "$2"\n')
    fake.chmod(0o755)
    lib, check = tmp_path / "libep.so", tmp_path / "_tensor_ptr.so"
    monkeypatch.setattr(hip_build, "HIPCC", str(fake))
    monkeypatch.setattr(hip_build, "CXX", str(fake))
    monkeypatch.setattr(hip_build, "LIB", str(lib))
    monkeypatch.setattr(hip_build, "TENSOR_PTR", str(check))
    other = tmp_path / "other.so"
    hip_build.build(lib=str(other), build_dir=str(tmp_path / "objects"))
    assert other.exists() and not check.exists()
    hip_build.build(lib=str(lib), build_dir=str(tmp_path / "objects"))
    assert lib.exists() and check.exists()
