"""What the compiler makes of the grouped products' variants that keep a tile's sums in registers: none may spill (the warp that
issues the MMAs would pay for it), whatever the kernel's other modes need."""
import os
import re
import subprocess

import pytest

from latent_moe_layer_gb300 import build

# mode (0 mm, 1 grad_x, 2 grad_w), output, rows that end inside 16 bytes, pairs a tile, parts added up in registers
VARIANTS = [("0, __nv_bfloat16, false, 1, true", 168), ("1, __half, false, 1, true", 168), ("0, float, false, 1, true", 168),
            ("0, __nv_bfloat16, false, 1, false", 96), ("2, __nv_bfloat16, false, 4, true", 96), ("2, float, false, 2, true", 96)]


@pytest.mark.skipif(not os.path.exists(build.NVCC), reason="needs nvcc")
def test_products_keep_their_sums_in_registers(tmp_path):
    src = tmp_path / "variants.cu"
    src.write_text('#include "group_tc.cuh"\n' +
                   "".join(f"void *variant_{i}() {{ return (void *)&k3::group_tc_kernel<{v}>; }}\n" for i, (v, _) in enumerate(VARIANTS)))
    r = subprocess.run([build.NVCC, *build.ARCH, *build.FLAGS, "-Xptxas", "-v", "-c", str(src), "-o", str(tmp_path / "variants.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    spills = re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", r.stderr)
    registers = sorted(int(n) for n in re.findall(r"Used (\d+) registers", r.stderr))
    assert len(spills) == len(registers) == len(VARIANTS)
    assert all(s == ("0", "0") for s in spills), r.stderr
    assert all(have <= want for have, want in zip(registers, sorted(n for _, n in VARIANTS)))
