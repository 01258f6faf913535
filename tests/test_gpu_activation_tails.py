"""The input gradient's activation derivative where it is small: blocks whose saved pre-activations are all strongly
negative, which take their INT8 scale from act' values far below 1.

Tolerances, fixed before the first run. act'(-x), x > 0, is a difference of two positive terms, the larger at least 3
times the other on the ranges tested, so a relative error eps of both is one of at most 2 eps of the result. Each term is
an exponential whose argument z carries a few fp32 roundings, which are absolute errors in the exponent:
  GELU       z = x^2 / 2: x = m s (counted twice: x^2), the constants and products of both exponents: 9 z 2^-24
  SiLU       z = x: x, log2 e and their product: 3 z 2^-24
  GELU-tanh  z = x (C0 + C1 x^2): x counts up to three times, five more roundings, log2 e and its product: 11 z 2^-24
Approximate exp2 (2 ulp), reciprocal (1 ulp), the erfc fit (1.2e-7) and the polynomial: 2^-20 together. The product
dY W here is one term: three roundings, inside the same 2^-20."""
import math

import pytest
import torch

import int8_fully_quantized_b200 as jf

import block_ref as B
from gpu_common import check_status

pytestmark = pytest.mark.gpu

EXPONENT = {"gelu": lambda x: 9 * x * x / 2, "silu": lambda x: 3 * x.abs(),
            "gelu_tanh": lambda x: 11 * 2 * math.sqrt(2 / math.pi) * (x.abs() + 0.044715 * x.abs() ** 3)}
# 1 / (1 + exp(-x)) and its square of the plain form lose nothing here: x < 0, sigmoid near 0; erfc is evaluated directly


def _grad(x, act):
    """act' in 64 bits without cancellation between numbers near 1 (block_ref.act_grad holds for x < 0)."""
    return B.act_grad(x, act)


@pytest.mark.parametrize("act,lo,hi", [("gelu", -5, -3), ("gelu", -7, -5), ("gelu", -12, -9), ("silu", -8, -4), ("silu", -18, -12),
                                       ("silu", -80, -60), ("gelu_tanh", -4, -2.5), ("gelu_tanh", -7, -5)])
@pytest.mark.parametrize("rows", [32, 160])
def test_derivatives_of_negative_blocks(act, lo, hi, rows):
    """dY = ones through W = I: Z = act'(P) for P in [lo, hi], dense and INT8, relative to act' itself."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    P = jf.QTensor(*B.quantize(torch.rand(rows, 64, generator=g, device="cuda") * (hi - lo) + lo))
    eye = jf.QTensor(*B.quantize(torch.eye(64, device="cuda")))
    ones = jf.QTensor(*B.quantize(torch.ones(rows, 64, device="cuda")))
    x = B.value(*P)
    want = (B.value(*ones) @ B.value(*eye)) * _grad(x, act)
    tol = 2 * (EXPONENT[act](x) * 2.0 ** -24 + 2.0 ** -20) * want.abs()
    z = jf.linear_dgrad_epilogue(ones, eye, P, act, out_dtype=torch.float32)
    assert ((z.double() - want).abs() <= tol + 2.0 ** -149).all()
    Z = jf.linear_dgrad_epilogue(ones, eye, P, act)
    q, s = B.quantize(want)
    rel = (tol / want.abs()).max().item()
    assert ((Z.s - s).abs() <= (rel + 2.0 ** -22) * s).all()
    # a code moves by one where the value lies within 127 * 2 rel of a tie
    d = (Z.q.int() - q.int()).abs()
    assert d.max() <= 1
    check_status()


@pytest.mark.parametrize("act", ["gelu", "silu", "gelu_tanh"])
def test_fused_and_separate_gradients_agree_in_the_tail(act):
    """One block in the tail beside blocks around 0: the tail's block has a scale of its own and keeps its digits."""
    P = torch.randn(64, 64, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    P[:32, :32] = torch.linspace(-6.5, -5.0, 1024, device="cuda").reshape(32, 32)
    P = jf.QTensor(*B.quantize(P))
    eye = jf.QTensor(*B.quantize(torch.eye(64, device="cuda")))
    ones = jf.QTensor(*B.quantize(torch.ones(64, 64, device="cuda")))
    Z = jf.linear_dgrad_epilogue(ones, eye, P, act)
    x = B.value(*P)[:32, :32]
    want = (B.value(*ones) @ B.value(*eye))[:32, :32] * _grad(x, act)
    got = B.value(*Z)[:32, :32]
    rel = 2 * (EXPONENT[act](x) * 2.0 ** -24 + 2.0 ** -20)
    # half a code of the block, its scale within rel
    assert ((got - want).abs() <= want.abs().max() / 127 * 0.5 * (1 + 127 * 2 * rel.max())).all()
    if act == "gelu":
        dY = jf.QTensor(*B.quantize(torch.ones(64, 64, device="cuda")))
        sep = B.value(*jf.gelu_i8_bwd(P, dY))[:32, :32]
        assert ((got - sep).abs() <= want.abs().max() / 127 * 1.01).all()
    check_status()
