"""The built kernels of the mixture-of-experts operators, read from the code
objects in the libraries (CPU; skipped when a library or a tool is missing):
none has a scratch segment (a spill's wait would also wait for the asynchronous
copies in flight), and the single-stage twin's weight gradient really is another
pipeline, with one LDS stage."""
import os
import re
import subprocess

import pytest

from moe_grouped_gemm_block_amd import build
from test_build_noscratch import MAGIC, TOOLS

EXPECTED = ("dg_moe_sort_one_i64", "dg_moe_sort_count_i32", "dg_moe_sort_place_i32", "dg_moe_permute_b2",
            "dg_moe_permute_fp8_bf16_pow2", "dg_moe_combine_bf16", "dg_moe_combine_bwd_bf16", "dg_swiglu_fp8_bf16",
            "dg_swiglu_fp8_bwd_bf16", "dg_wgrad256_f32", "dg_wgrad128_bf16")


def kernel_notes(lib, tmp):
    """{kernel: {field: bytes}} of the fixed segment sizes in a library's code objects."""
    if not os.path.exists(lib):
        pytest.skip(f"{lib} is not built")
    for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-readelf"):
        if not os.path.exists(os.path.join(TOOLS, t)):
            pytest.skip(f"{t} not found")

    def tool(name, *args):
        return subprocess.run([os.path.join(TOOLS, name), *args], check=True, capture_output=True, text=True).stdout

    fat, part, co = (str(tmp / n) for n in ("fat", "part", "co"))
    tool("llvm-objcopy", f"--dump-section=.hip_fatbin={fat}", lib, str(tmp / "copy"))
    data = open(fat, "rb").read()
    starts = [m.start() for m in re.finditer(re.escape(MAGIC), data)] + [len(data)]
    out = {}
    for a, b in zip(starts, starts[1:]):
        open(part, "wb").write(data[a:b])
        tool("clang-offload-bundler", "--unbundle", "--type=o", f"--input={part}",
             "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--output={co}")
        sizes = {}
        for line in tool("llvm-readelf", "--notes", co).splitlines():
            m = re.match(r"\s+\.(group|private)_segment_fixed_size:\s+(\d+)", line)
            if m:
                sizes[m.group(1)] = int(m.group(2))
            m = re.match(r"\s+\.symbol:\s+(\S+)\.kd", line)
            if m:
                out[m.group(1)], sizes = sizes, {}
    return out


def named(notes, name):
    """The sizes of the one kernel dg::name."""
    found = [v for k, v in notes.items() if f"{len(name)}{name}E" in k]
    assert len(found) == 1, (name, len(found))
    return found[0]


def test_no_kernel_has_scratch(tmp_path):
    notes = kernel_notes(build.LIB, tmp_path)
    for name in EXPECTED:
        named(notes, name)
    ours = {k: v for k, v in notes.items() if re.search(r"dg_(moe|swiglu|wgrad)", k)}
    assert len(ours) >= 26
    assert not {k: v for k, v in ours.items() if v["private"] != 0}


@pytest.mark.parametrize("kernel", ["dg_wgrad256_bf16", "dg_wgrad256_f32", "dg_wgrad128_bf16", "dg_wgrad128_f32"])
def test_single_stage_weight_gradient(tmp_path, kernel):
    sizes = [named(kernel_notes(lib, tmp_path), kernel)["group"] for lib in (build.LIB, build.LIB_STAGES1)]
    assert 2 * sizes[1] <= sizes[0], sizes
