"""gelu and its slope relative to their values, down to where they leave the type's normal range, and
how silu's own gradient is rounded.

Phi(-|z|) is computed as exp(-z^2 / 2) times a function of |z|, in fp32.  Relative errors for |z|
up to 13: the function's fit 3e-9; eleven multiply-adds and two products, each half a step (2^-24),
and a quotient, a whole one with at most twice the weight, 17 * 2^-24 = 1.01e-6; 2^x a step, 1.2e-7;
the argument z^2 log2(e) / 2 <= 122 is off by its constant's and its product's half steps (z^2 of a
16-bit z is exact), 122 * ln 2 * 2 * 2^-24 = 1.01e-5.  Together 1.13e-5, below 2^-16 = 1.53e-5.
The slope Phi(z) + z phi(z) adds two terms that are each that close, and rounds
once more: 2^-16 of the sum of their magnitudes."""
import math

import pytest
import torch

from combine_moe_layout_amd import binding as B
from products_ref import TYPES, half_step

pytestmark = pytest.mark.gpu
REL = 2.0 ** -16


def every_value(dt, lo, hi):
    """All values of a 16-bit type in [lo, hi], padded with zeros to whole rows of 64."""
    v = torch.arange(-2 ** 15, 2 ** 15, device="cuda", dtype=torch.int32).to(torch.int16).view(dt)
    v = v[torch.isfinite(v) & (v >= lo) & (v <= hi)]
    return torch.cat([v, v.new_zeros(-v.numel() % 64)]).reshape(-1, 64)


def parts(z):
    """Phi(z) and z phi(z) in 64 bits."""
    return 0.5 * torch.erfc(-z * math.sqrt(0.5)), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def close(got, ref, before, what):
    tol = before + half_step(ref.abs() + before, got.dtype)
    worst = ((got.double() - ref).abs() / tol).max().item()
    assert worst <= 1.0, "%s: %.3g of the tolerance" % (what, worst)


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("times", [1, 40, 600])
def test_gelu_of_every_value(name, times):
    """Through a product with the identity, which is exact (rows for each of the kernels)."""
    print("[gpu-activations] forward", name, times, flush=True)
    dtype, dt = TYPES[name]
    x = every_value(dt, -13.0, 13.0).repeat(times, 1)
    eye = torch.eye(64, device="cuda").to(dt)
    out, pre = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    B.ep_linear(x, eye, out, dtype, act=B.EP_ACT_GELU, preact=pre)
    assert torch.equal(pre, x)
    z = x.double()
    ref = z * parts(z)[0]
    close(out, ref, REL * ref.abs(), "gelu")


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("times", [0, 1, 40, 600])
def test_gelu_slope_of_every_value(name, times):
    """ep_act_grad (times 0), and the rows' gradient of a product with the identity."""
    print("[gpu-activations] slope", name, times, flush=True)
    dtype, dt = TYPES[name]
    z16 = every_value(dt, -13.0, 13.0).repeat(max(times, 1), 1)
    d = torch.ones_like(z16)
    d[:, ::3] = -1.5
    dz = torch.full_like(z16, 7.0)
    if times:
        n = 256 if times == 1 else 64      # a longer reduction takes the kernel whose waves share it
        dy, w = d.new_zeros((d.shape[0], n)), d.new_zeros((n, 64))
        dy[:, :64], w[:64] = d, torch.eye(64, device="cuda")
        B.ep_linear_grad_x(dy, w, dz, dtype, act=B.EP_ACT_GELU, preact=z16)
    else:
        B.ep_act_grad(d, z16, dz, dtype, B.EP_ACT_GELU)
    cdf, bell = parts(z16.double())
    close(dz, d.double() * (cdf + bell), REL * d.double().abs() * (cdf + bell.abs()), "slope")


@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_gelu_with_more_columns_than_rows(name):
    """The kernel for few rows: values along the columns, from the bias alone."""
    print("[gpu-activations] few rows", name, flush=True)
    dtype, dt = TYPES[name]
    bias = every_value(dt, -13.0, 13.0).reshape(-1)
    N = bias.numel()
    x, w = torch.zeros((3, 8), dtype=dt, device="cuda"), torch.zeros((N, 8), dtype=dt, device="cuda")
    out = torch.full((3, N), 7.0, dtype=dt, device="cuda")
    B.ep_linear(x, w, out, dtype, act=B.EP_ACT_GELU, bias=bias)
    z = bias.double()
    ref = z * parts(z)[0]
    for r in range(3):
        close(out[r], ref, REL * ref.abs(), "row %d" % r)


@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_silu_gradient_rounds_as_its_formula(name):
    """ep_act_grad through silu gives the bits of the formula in fp32 operations, each rounded."""
    print("[gpu-activations] silu", name, flush=True)
    dtype, dt = TYPES[name]
    z = every_value(dt, -60.0, 60.0).repeat(8, 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    d = torch.randn(z.shape, device="cuda", generator=g).to(dt)
    dz = torch.full_like(z, 7.0)
    B.ep_act_grad(d, z, dz, dtype, B.EP_ACT_SILU)
    p = 1 / (1 + torch.exp(-z.float()))
    assert torch.equal(dz, (d.float() * p * (1 + z.float() * (1 - p))).to(dt))
