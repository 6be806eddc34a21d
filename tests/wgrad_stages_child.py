"""Child process of tests/test_gpu_wgrad_stages.py (not collected by pytest):
weight gradients through the library named by DG_LIBRARY, their raw bytes saved
to the .npz file named on the command line."""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from moe_grouped_gemm_block_amd import dg  # noqa: E402

DEV = "cuda:0"
# rows of each expert, N, K: even and uneven experts, one row, no rows, part tiles,
# 128- and 256-row tiles (the second from more than 256 tiles on), many steps
CASES = {"one_row": ([1], 8, 16), "parts": ([0, 33, 1, 0, 64], 136, 144), "steps": ([300, 31, 65, 2048], 520, 272),
         "even": ([256] * 8, 1024, 1024), "even_256": ([160] * 5, 2048, 1024), "uneven_256": ([700, 0, 5, 64, 33], 2048, 1040)}


def main():
    print(f"weight gradient stages child: {os.path.basename(dg.LIB_PATH)}", flush=True)
    res = {}
    for i, (name, (rows, N, K)) in enumerate(CASES.items()):
        print(f"  {name}", flush=True)
        g = torch.Generator(device=DEV).manual_seed(i)
        M = sum(rows)
        offs = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=DEV)
        slot_row = torch.arange(M, dtype=torch.int32, device=DEV)
        x, sx = dg.moe_permute_fp8(torch.randn(M, K, device=DEV, generator=g), slot_row[:, None].contiguous(), slot_row)
        dy = torch.randn(M, N, device=DEV, generator=g).bfloat16()
        for out in ("f32", "bf16"):
            dw = dg.grouped_wgrad_fp8(dy, x, sx, offs, out_dtype=out)
            res[f"{name}_{out}"] = dw.view(torch.uint8).cpu().numpy().copy()
            dw = dg.grouped_wgrad_fp8(dy, x, sx, offs, out_dtype=out, dW=dw, accumulate=True)
            res[f"{name}_{out}_twice"] = dw.view(torch.uint8).cpu().numpy().copy()
    np.savez(sys.argv[1], **res)
    print(f"  saved {len(res)} outputs", flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
