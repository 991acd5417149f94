"""Rows to 8-bit integers at the sizes between which a row's lanes change."""
import pytest
import torch

import test_gpu_int8 as int8
from combine_moe_layout_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [3, 16383, 16384, 16391])
@pytest.mark.parametrize("n", [1024, 1040, 2048, 2064, 3056, 3088, 4096])
def test_rows_of_each_width(rows, n):
    print("[gpu-int8] width", rows, n, flush=True)
    x = torch.randn((rows, n), device="cuda", generator=int8.gen(rows + n)).to(torch.bfloat16)
    x[rows // 2, n - 1], x[rows - 1] = float("nan"), 0
    q = torch.full((rows, n), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), 7.0, device="cuda")
    B.ep_quantize_int8(x, q, s, B.EP_BF16)
    int8.same_rows(q, s, x)
