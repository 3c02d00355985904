"""The Python binding of the norm and the feed-forward block: what it refuses before the library sees it, and what it
asks of torch (no GPU needed)."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_aux_b200 import binding
    binding.load()
    return binding


def test_sizes_past_32_bits_are_refused(B):
    """2^32 + 4 rows would be four rows to the library."""
    T = 2 ** 32 + 4
    with pytest.raises(ValueError, match="32 bits"):
        B.moe_rmsnorm_bwd_workspace_size(T, 8)
    with pytest.raises(ValueError, match="32 bits"):
        B.moe_rmsnorm_bwd_workspace_size(4, 2 ** 32 + 8)
    for n in ("T", "H", "F"):
        with pytest.raises(ValueError, match="32 bits"):
            B.make_ffn_config(**{**dict(T=4, H=8, F=8), n: 2 ** 32 + 8})
    # a tensor of that many rows, of one row's memory, as the norm's x and h
    x = torch.zeros(8, dtype=torch.bfloat16).expand(T, 8)
    with pytest.raises(ValueError, match="32 bits"):
        B.moe_rmsnorm_fwd(x, None, x[0], 1e-5, None, x, None, None, None)
    with pytest.raises(ValueError, match="32 bits"):
        B.moe_rmsnorm_bwd(x, x, x[0], None, None, x, None, None)
    # the largest that fit pass the binding (the library then refuses by its own rules, or not)
    assert B.moe_rmsnorm_bwd_workspace_size(2 ** 31 - 1, 8) == 296 * 8 * 4 + (-(296 * 8 * 4)) % 256
    assert B.make_ffn_config(T=2 ** 31 - 1, H=8, F=8).T == 2 ** 31 - 1


def python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_a_torch_without_cuda_is_enough_for_the_refusals():
    """A build of torch without CUDA has none of these names."""
    python("""
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    delattr(torch._C, name)
from mixture_experts_layer_aux_b200 import binding as b
assert b.load().moe_rmsnorm_fwd(0, 8, None, None, None, 1e-5, None, None, None, None, None, None) == 1
assert b.moe_ffn_workspace_size(b.make_ffn_config(1, 64, 64)) > 0
""")


def test_package_names_follow_the_binding():
    """A name of the package is the binding's at that time: the library once it is loaded, and what a caller put there."""
    python("""
import mixture_experts_layer_aux_b200 as moe
assert moe._lib is None
moe.load()
assert moe._lib is not None
from mixture_experts_layer_aux_b200 import binding
assert moe.moe_ffn_saved_size is binding.moe_ffn_saved_size
binding.moe_ffn_saved_size = len
assert moe.moe_ffn_saved_size is len
""")


def test_package_keeps_its_own_names():
    """What is bound anew in the binding takes nothing from the package that is the package's own."""
    python("""
import mixture_experts_layer_aux_b200 as moe
from mixture_experts_layer_aux_b200 import binding
own = moe.load
binding.load = binding.load
assert moe.load is own
f = moe.moe_ffn_saved_size
binding.moe_ffn_saved_size = len
binding.moe_ffn_saved_size = f
assert moe.moe_ffn_saved_size is f and vars(moe)["moe_ffn_saved_size"] is f
""")
