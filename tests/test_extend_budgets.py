"""Register budgets of the extend kernels by type, head size and tile height, read
from the compiler's resource report on the CPU: what each must stay under for as
many CTAs to share an SM as its shared memory lets.

65536 registers, handed out to warps in steps of 256: R registers a thread take
ceil(32 R / 256) * 256 of a warp.
"""
import pytest

from tests.test_kernel_resources import _resources


def ctas(regs, threads):
    return 65536 // (-(-32 * regs // 256) * 256 * (threads // 32))


def test_the_rule():
    assert ctas(168, 128) == 3 and ctas(169, 128) == 2 and ctas(184, 128) == 2
    assert ctas(168, 192) == 2 and ctas(176, 192) == 1 and ctas(96, 128) == 5


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tensor_core_kernels(dtype, D):
    found = {k: v for k, v in _resources(f"extend_tc_{dtype}_d{D}.cu").items() if "extend_tc_kernel" in k}
    assert len(found) == (6 if D == 128 else 4)
    for name, (regs, spill) in found.items():
        tall = "Li128ELi2E" in name
        # one CTA of 352 threads (allotted like 384), two of 192, or with 512-byte rows one of 192
        assert ctas(regs, 384 if tall else 192) >= (1 if tall or D == 256 else 2), (name, regs)
        assert spill == 0, (name, spill)


def test_cuda_core_kernels():
    found = {k: v for k, v in _resources("extend_fma_f32.cu").items() if "extend_fma_kernel" in k}
    # shared memory lets three CTAs of 64 x 64 tiles share an SM and two of 128-wide rows
    want = {"ILi64ELi64E": 3, "ILi128ELi64E": 2, "ILi64ELi16E": 5, "ILi128ELi16E": 2}
    assert len(found) == len(want)
    for shape, least in want.items():
        (regs, spill), = [v for k, v in found.items() if shape in k]
        assert ctas(regs, 128) >= least and spill == 0, (shape, regs, spill)
