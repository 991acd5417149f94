"""The products and gradients at the ends of what their header allows."""
import pytest
import torch

from combine_moe_layout_amd import binding as B
from products_ref import SUM, check

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("T", [2 ** 25 - 1, 2 ** 31 - 1])
def test_weights_gradient_of_the_most_rows(T):
    """All rows are zero but 100 at both ends, so the sums are those of 200 rows.  (A workgroup walks
    all rows of its tile: the larger case is seconds of one kernel.)"""
    if torch.cuda.mem_get_info()[0] < T * 16 + 2 ** 30:
        pytest.skip("needs %d GB" % (T >> 26))
    print("[gpu-products-edges] rows", T, flush=True)
    x = torch.zeros((T, 8), dtype=torch.bfloat16, device="cuda")
    ends = torch.randn((200, 8), device="cuda", generator=gen(1)).to(torch.bfloat16)
    x[:100], x[-100:] = ends[:100], ends[100:]
    dw, db = torch.full((8, 8), 7.0, device="cuda"), torch.full((8,), 7.0, device="cuda")
    B.ep_linear_grad_w(x, x, dw, B.EP_BF16 | B.EP_GRAD_F32, dbias=db)   # both operands may be one tensor
    torch.cuda.synchronize()
    e = ends.double()
    check(dw, e.T @ e, 200 * SUM * (e.abs().T @ e.abs()), "dweights")
    check(db, e.sum(0), 200 * SUM * e.abs().sum(0), "dbias")
    del x
    torch.cuda.empty_cache()


def test_one_expert_with_the_largest_capacity():
    """A few rows in a padded buffer of 2^31 - 1: the grid follows the rows wanted, not the capacity."""
    cap = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 3 * cap * 16 + 2 ** 30:
        pytest.skip("needs 104 GB")
    print("[gpu-products-edges] capacity", cap, flush=True)
    g = gen(2)
    lay = B.EpLayout(5, 1, 1, 1, cap)
    B.ep_get_layout(torch.zeros((5, 1), dtype=torch.int64, device="cuda"), lay)
    x, out = (torch.empty((cap, 8), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[:5] = torch.randn((5, 8), device="cuda", generator=g).to(torch.bfloat16)
    out[:8] = 7.0
    w = torch.randn((1, 8, 8), device="cuda", generator=g).to(torch.bfloat16)
    B.ep_expert_gemm(x, w, lay, out, B.EP_BF16)
    dx = torch.empty_like(out)
    dx[:8] = 7.0
    B.ep_expert_gemm_grad_x(x, w, lay, dx, B.EP_BF16)
    torch.cuda.synchronize()
    v, m = x[:5].double(), w[0].double()
    check(out[:5], v @ m.T, 8 * SUM * (v.abs() @ m.abs().T), "out")
    check(dx[:5], v @ m, 8 * SUM * (v.abs() @ m.abs()), "dx")
    assert (out[5:8] == 7).all() and (dx[5:8] == 7).all()
    del x, out, dx
    torch.cuda.empty_cache()
