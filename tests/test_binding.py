"""What the binding needs to load and to be built, and its answers to missing arguments. Every
call here fails a check or asks only for sizes: no kernel is launched."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import combine_ep_get_03_amd as ep
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


T, H, K = 4, 256, 2
X = torch.zeros((T, H), dtype=torch.bfloat16)
W = torch.ones(H)
SLOT = torch.zeros((T, K), dtype=torch.int32)
ROWS = torch.zeros((T * K, H), dtype=torch.bfloat16)
C8, S8 = torch.zeros((T, H), dtype=torch.uint8), torch.ones((T, H // 128))
P8, PS = torch.zeros((T * K, H), dtype=torch.uint8), torch.ones((T * K, H // 128))
CALLS = {
    "ep_rmsnorm": (ep.ep_rmsnorm, dict(x=X, weight=W, y=X)),
    "ep_rmsnorm_grad": (ep.ep_rmsnorm_grad, dict(h=X, weight=W, grad_y=X, grad_x=X)),
    "ep_dispatch_permute_fp8": (ep.ep_dispatch_permute_fp8,
                                dict(x_fp8=C8, x_scales=S8, topk_weights=None, expert_slot=SLOT,
                                     perm_x_fp8=P8, perm_scales=PS)),
    "ep_combine_unpermute": (ep.ep_combine_unpermute,
                             dict(expert_out=ROWS, topk_weights=None, expert_slot=SLOT, out=X)),
    "ep_combine_unpermute_grad": (ep.ep_combine_unpermute_grad,
                                  dict(grad_out=X, expert_out=None, topk_weights=None,
                                       expert_slot=SLOT, grad_expert_out=ROWS)),
    "ep_dispatch_permute_grad": (ep.ep_dispatch_permute_grad,
                                 dict(grad_perm_x=ROWS, expert_slot=SLOT, grad_x=X)),
}


@pytest.mark.parametrize("name,arg", [
    ("ep_rmsnorm", "x"), ("ep_rmsnorm", "weight"), ("ep_rmsnorm_grad", "h"),
    ("ep_rmsnorm_grad", "weight"), ("ep_dispatch_permute_fp8", "x_fp8"),
    ("ep_dispatch_permute_fp8", "expert_slot"), ("ep_dispatch_permute_fp8", "perm_x_fp8"),
    ("ep_combine_unpermute", "expert_out"), ("ep_combine_unpermute", "expert_slot"),
    ("ep_combine_unpermute_grad", "grad_out"), ("ep_combine_unpermute_grad", "expert_slot"),
    ("ep_combine_unpermute_grad", "grad_expert_out"), ("ep_dispatch_permute_grad", "grad_perm_x"),
    ("ep_dispatch_permute_grad", "expert_slot")])
def test_a_missing_tensor_is_named(name, arg):
    """The arguments that a call looks at before it takes any address."""
    call, args = CALLS[name]
    with pytest.raises(ValueError, match=f"^{arg} is required"):
        call(**{**args, arg: None})
    for value in ([1.0], 5, np.ones((T, H))):
        with pytest.raises(TypeError, match=f"^{arg}: expected a tensor"):
            call(**{**args, arg: value})


def test_codes_that_are_no_tensor_are_refused():
    codes = _binding._codes_ptr
    assert codes(None, (T, H), "y_fp8", 0, False) is None
    for value in ([1], 5, np.zeros((T, H), np.uint8)):
        with pytest.raises(TypeError, match="y_fp8: expected a tensor"):
            codes(value, (T, H), "y_fp8", 0, False)
    with pytest.raises(ValueError, match="y_fp8 is required"):
        codes(None, (T, H), "y_fp8", 0)
    with pytest.raises(TypeError, match="weight: expected torch.bfloat16 or torch.float32"):
        ep.ep_rmsnorm(X, W.half(), y=X)


@pytest.mark.gpu
def test_a_workspace_that_is_no_tensor_is_refused():
    """Refused by the binding, with every other argument in order: nothing is launched."""
    x, w = X.cuda(), W.cuda()
    out = torch.full_like(x, 3.0)
    for value in ([0], 5, np.zeros(1 << 16, np.uint8)):
        with pytest.raises(TypeError, match="workspace: expected a tensor"):
            ep.ep_rmsnorm_grad(x, x, w, grad_x=out, workspace=value)
    with pytest.raises(TypeError, match="workspace: expected torch.uint8"):
        ep.ep_rmsnorm_grad(x, x, w, grad_x=out, workspace=w)
    assert torch.all(out == 3.0)
