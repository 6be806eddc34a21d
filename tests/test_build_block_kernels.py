"""The built kernels of the router, the norms around a block and clipping, read from the
code objects in the library (CPU; skipped when a library or a tool is missing): they are
there, and none has a scratch segment."""
import re

from moe_grouped_gemm_block_amd import build
from test_build_moe_kernels import kernel_notes, named


def test_no_kernel_has_scratch(tmp_path):
    notes = kernel_notes(build.LIB, tmp_path)
    for name in ("dg_moe_route_f32_16x4", "dg_moe_route_bf16_64x16_bias", "dg_moe_route_bwd_bf16_16x16",
                 "dg_moe_route_finish", "dg_residual_norm_columns", "dg_grad_squares", "dg_grad_norm_sum",
                 "dg_clip_scale"):
        named(notes, name)
    ours = {k: v for k, v in notes.items() if re.search(r"dg_(moe_route|residual_norm|grad|clip)", k)}
    assert sum("residual_norm_kernel" in k for k in ours) >= 16
    assert sum("residual_norm_bwd_kernel" in k for k in ours) >= 16
    assert not {k: v for k, v in ours.items() if v["private"] != 0}
