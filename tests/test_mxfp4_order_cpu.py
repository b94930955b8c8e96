"""The both-forms quantiser's exchange of row scales through LDS, in the device IR as the
front end emits it: 16 lanes store two scales each and every one of them reads all 32, so the
store and the reads need an order that no optimisation may undo."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from precision_dense_gemm_amd import build

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCE = next(s for s in build.SOURCES if s.endswith("mxfp4.hip"))


@pytest.fixture(scope="module")
def ir(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    out = str(tmp_path_factory.mktemp("ir") / "mxfp4.ll")
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    subprocess.run([HIPCC, *flags, "-I", build.INCLUDE, "--cuda-device-only", "-S", "-emit-llvm", "-Xclang",
                    "-disable-llvm-passes", SOURCE, "-o", out], check=True, capture_output=True, timeout=300)
    with open(out) as f:
        return f.read()


@pytest.mark.parametrize("type_", [0, 1, 2], ids=["f32", "f16", "bf16"])
def test_row_scales_are_ordered_between_lanes(ir, type_):
    start = re.search(rf"^define amdgpu_kernel void @\S*mx_quant_cols_kernelILi{type_}ELb1E", ir, re.M).start()
    body = ir[start:ir.index("\n}\n", start)]
    # from the first use of the scales' LDS to the workgroup's barrier
    exchange = body[body.index("E3scr"):body.index("@_Z13__syncthreadsv")]
    calls = [m for m in re.finditer(r"call void @(\S*wave_lds_order\S*)\(\)", exchange)]
    assert len(calls) == 1, "no order between the lanes' stores and reads"
    order = ir[ir.index(f"define internal void @{calls[0][1]}()"):]
    assert re.findall(r"fence syncscope\(\"wavefront\"\) \w+|@llvm\.amdgcn\.wave\.barrier", order[:order.index("\n}\n")]) == [
        'fence syncscope("wavefront") release', "@llvm.amdgcn.wave.barrier", 'fence syncscope("wavefront") acquire']
    before, after = exchange[:calls[0].start()], exchange[calls[0].end():]
    # both sides as bytes: accesses of two types would be taken not to overlap, fence or not
    copies = r"@llvm\.memcpy\.\S+\(.*?, i64 (\d+), i1 false\)"
    assert re.findall(copies, before) == ["2"] and re.findall(copies, after)[:1] == ["32"]
