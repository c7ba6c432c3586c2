"""Plans of the MXFP4 products over sizes, layouts and types, on the CPU: each is of a kernel that is built."""
import torch

import dense_gemm_19_amd as dg

F16, BF16, I32, U8 = torch.float16, torch.bfloat16, torch.int32, torch.uint8
E = 4


def test_plans_have_kernels():
    # over sizes, layouts and types: tiles of codes larger than 64 never meet K in pieces, and the kernels of 16-bit rows
    # between few and many have 32 or 48 of them (no others are built)
    for rows in (1, 5, 16, 17, 20, 32, 33, 37, 48, 49, 64, 65, 97, 128, 129, 150, 193, 300, 700, 1030, 2100, 4000):
        for cols in (33, 300, 1000, 2900, 4096, 4200, 8200):
            for k in (30, 96, 333, 1024, 4100, 9000):
                q, s, c = torch.empty(cols, (k + 1) // 2, dtype=U8), torch.empty(cols, -(-k // 32), dtype=U8), torch.empty(rows, cols, dtype=BF16)
                for a, sa in ((torch.empty(rows, k, dtype=F16), None), (torch.empty(rows, (k + 1) // 2, dtype=U8), torch.empty(rows, -(-k // 32), dtype=U8))):
                    plan = dg.gemm_mx4_plan(a, q, s, c, SA=sa)
                    for part in plan.split("; "):
                        if "loads" in part and "64x64" not in part:
                            assert "K in 1 pieces" in part, (rows, cols, k, plan)
                        if part.startswith(("aligned words", "any layout")):
                            assert " 32x64" in part or " 48x64" in part, (rows, cols, k, plan)
                off, q3, s3 = torch.empty(E + 1, dtype=I32), q[None].expand(E, -1, -1), s[None].expand(E, -1, -1)
                plan = dg.moe_gemm_mx4_plan(torch.empty(rows, k, dtype=BF16), off, q3, s3, c)
                assert not plan.startswith(("aligned words", "any layout")) or " 32x64" in plan or " 48x64" in plan, (rows, cols, k, plan)
