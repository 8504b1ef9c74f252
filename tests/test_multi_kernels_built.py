"""Every kernel of the multi-adapter calls and of the AdamW step is in the built library (that
none of them uses scratch memory or spills is checked for all kernels together)."""
import pytest

from test_kernel_resources import _kernels

KERNELS = ["multi_plan_kernel", "multi_prologue_kernelILi1E", "multi_prologue_kernelILi8E", "multi_reduce_small", "skinny_nf4ILi4ELb1E",
           "gemv_nf4_kernelILi1ELb1ELb1E", "gemv_nf4_persistILi1ELb1ELb0ELb1E", "multi_grad_mfmaILi1E", "multi_grad_mfmaILi2E",
           "multi_grad_reduce", "gemm_multi_reduce", "adamw_kernel", "adamw_moments_kernel"]
KERNELS += [f"gemm_multi_{form}{dx}" for form in ("kernel", "split", "mixed", "half", "half_split") for dx in ("E", "_dxE")]


def test_built(tmp_path):
    names = [k[".name"] for k in _kernels(tmp_path)]
    missing = [e for e in KERNELS if not any(e in n for n in names)]
    assert not missing, missing
