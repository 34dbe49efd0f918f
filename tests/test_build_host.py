"""The build's check of the compiler's register report."""
import os
import subprocess

import pytest

from lossless_entropy_coding_amd import build

KERNEL = """x.hip:1:0: remark: Function Name: {name} [-Rpass-analysis=kernel-resource-usage]
x.hip:1:0: remark:     VGPRs: {v} [-Rpass-analysis=kernel-resource-usage]
x.hip:1:0: remark:     AGPRs: {a} [-Rpass-analysis=kernel-resource-usage]
"""


def test_kernels_with_accumulation_registers_are_refused():
    good = KERNEL.format(name="first", v=240, a=0) + KERNEL.format(name="second", v=12, a=0)
    build.check_registers("x.hip", good)
    with pytest.raises(RuntimeError, match=r"x.hip.*third \(16\)"):
        build.check_registers("x.hip", good + KERNEL.format(name="third", v=256, a=16))
    build.check_registers("x.hip", "", kernels=False)
    for silent in ("", "x.hip:1:0: warning: unused", good + "x.hip:1:0: remark: Function Name: fourth"):
        with pytest.raises(RuntimeError, match="reported"):
            build.check_registers("x.hip", silent)


def test_the_compiler_reports_them(tmp_path):
    """One kernel with bounds that leave it two waves per SIMD, and with a bound of one, where results go to AGPRs."""
    src = tmp_path / "k.hip"
    src.write_text("""
#include <hip/hip_runtime.h>
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
__global__ __launch_bounds__(64, BOUND) void KERNEL(const bf16x8* x, f32x16* y, int n) {
    f32x16 acc[2] = {y[0], y[1]};
    for (int k = 0; k < n; k++)
        for (int i = 0; i < 2; i++) acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[k], x[k + i], acc[i], 0, 0, 0);
    for (int i = 0; i < 2; i++) y[i] = acc[i];
}
""")
    for name, bound, fits in (("bound_kernel", 2, True), ("free_kernel", 1, False)):
        r = subprocess.run([build.hipcc(), *build.HIP_FLAGS, f"-DKERNEL={name}", f"-DBOUND={bound}", "-c", str(src), "-o",
                            os.devnull, build.REPORT], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        if fits:
            build.check_registers("k.hip", r.stderr)
        else:
            with pytest.raises(RuntimeError, match=name):
                build.check_registers("k.hip", r.stderr)
