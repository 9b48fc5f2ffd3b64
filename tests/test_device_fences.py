"""Ordering of LDS traffic between lanes of one wave, in the device code as the front end emits it (no GPU).

Lanes that write LDS and other lanes of the wave that read it without a barrier in between need a fence:
nothing else keeps the compiler from moving the reads up, all the more since the two sides access
the bytes as different types."""
import os
import re
import subprocess

from block_scaled_fp4_05_amd import build

KERNEL = re.compile(r"^define amdgpu_kernel void @(\S*k_gemm8_tileI\S*Lb1EEEv\S*)\(.*?^}", re.M | re.S)   # bf16 output


def test_tile_product_orders_its_output_rows(tmp_path):
    out = str(tmp_path / "gemm8.ll")
    subprocess.run([build.hipcc(), *build.CXXFLAGS, "--cuda-device-only", "-S", "-emit-llvm", "-Xclang",
                    "-disable-llvm-passes", os.path.join(build.CSRC, "fp4q_gemm8.hip"), "-o", out],
                   check=True, capture_output=True)
    with open(out) as f:
        kernels = list(KERNEL.finditer(f.read()))
    assert len(kernels) >= 4
    for k in kernels:
        body = k.group(0)
        written = [m.end() for m in re.finditer(r"^\s+store i16 ", body, re.M)]   # two rows' halves, then the ragged tail
        converts = [m.end() for m in re.finditer(r"bf16_pair", body)]
        read = re.search(r"load <4 x i32>", body[converts[0]:])
        fence = re.search(r"wave_lds_fence", body[converts[0]:])
        assert len(written) >= 3 and read and fence, k.group(1)
        at, loads = converts[0] + fence.start(), converts[0] + read.start()
        assert written[1] < at < loads, k.group(1)
