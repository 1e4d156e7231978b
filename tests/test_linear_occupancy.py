"""The workgroups of the prompt walk that a CU holds: what lin_attn_prefill's segment lengths assume against the
registers and LDS of the built kernels.

The assumption shows in the workspace: one sequence that is long enough has one segment for each workgroup that the
chip holds, up to whole numbers, and one place more.  What the kernels use stands in their metadata (llvm-readelf
--notes): a SIMD has 512 registers a lane, given out by 8, and at most 8 waves; a CU has 4 SIMDs and 160 KiB of LDS.
"""
import os
import re
import subprocess
import tempfile

import pytest

import bench
import gated_deltanet_recurrent_decode_amd as gdn
from tests.test_machine_code import LIB, READELF


def _metadata():
    out = {}
    with tempfile.TemporaryDirectory() as d:
        for i, co in enumerate(bench.device_code_objects(LIB)):
            path = os.path.join(d, f"co{i}.elf")
            with open(path, "wb") as f:
                f.write(co)
            notes = subprocess.run([READELF, "--notes", path], capture_output=True, text=True, check=True).stdout
            for kernel in re.split(r"\n\s+- \.agpr_count:", notes)[1:]:
                name = re.search(r"\.name:\s+(\S+)", kernel).group(1)
                out[name] = {k: int(re.search(rf"\.{k}:\s+(\d+)", kernel).group(1))
                             for k in ("vgpr_count", "group_segment_fixed_size", "max_flat_workgroup_size")}
    return out


def test_walks_a_cu():
    if not os.path.exists(LIB) or not os.path.exists(READELF):
        pytest.skip("libgdn.so is not built, or there is no llvm-readelf")
    kernels = {n: m for n, m in _metadata().items() if "lin_prefill_kernel" in n}
    assert len(kernels) == 12, sorted(kernels)
    for (d_k, d_v, pair) in ((64, 64, 1), (64, 64, 2), (64, 128, 1), (128, 64, 1), (128, 64, 2), (128, 128, 1)):
        (m,) = [m for n, m in kernels.items() if f"ILi{d_k}ELi{d_v}ELi{pair}ELb1E" in n]
        waves = m["max_flat_workgroup_size"] // 64
        by_registers = min(8, 512 // (-(-m["vgpr_count"] // 8) * 8)) * 4 // waves
        holds = min(by_registers, 160 * 1024 // m["group_segment_fixed_size"])
        H_v = 16 * pair  # 16 workgroups a segment
        need = gdn.lin_attn_prefill_workspace_bytes(1, 20000, H_v // pair, H_v, d_k, d_v)
        segments = (need - 256) // (H_v * (d_k * d_v + 1) * 4) - 1
        assert segments == 256 * holds // 16, (d_k, d_v, pair, m, segments)
