"""Infinities and NaN through the activations of the linear epilogues: they reach the outputs by the activations'
formulas, so that a diverged product does not turn into ordinary numbers. They enter by the bias (an empty contraction)."""
import pytest
import torch

import int8_fully_quantized_b200 as jf

from gpu_common import check_status

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _forward(act, values, out_dtype=torch.float32, residual=None):
    bias = torch.linspace(-3, 3, 64, device="cuda")
    bias[:len(values)] = torch.tensor(values, device="cuda")
    return jf.linear_fwd_epilogue(jf.empty_qtensor(32, 0), jf.empty_qtensor(64, 0), bias, act, residual, out_dtype=out_dtype)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_relu_of_nan_and_infinities(dt):
    y = _forward("relu", [NAN, INF, -INF], dt)
    assert torch.isnan(y[:, 0]).all() and (y[:, 1] == INF).all() and (y[:, 2] == 0).all()
    assert torch.isfinite(y[:, 3:]).all()
    r = torch.ones(32, 64, device="cuda", dtype=dt)
    assert torch.isnan(_forward("relu", [NAN], dt, r)[:, 0]).all()
    # the codes, by the rules that hold without an activation: a block whose other values are all 0 has scale 0 and
    # codes 0 (columns 0..31 are not positive); in any other block the NaN gets -127 and the rest is unchanged
    Y, Z = _forward("relu", [NAN], None), _forward("relu", [0.0], None)
    assert torch.equal(Y.q, Z.q) and torch.equal(Y.s, Z.s) and not Y.s[:, 0].any()
    at40 = torch.linspace(-3, 3, 64).tolist()[:40]
    Y, Z = _forward("relu", at40 + [NAN], None), _forward("relu", at40 + [0.0], None)
    assert (Y.q[:, 40] == -127).all() and torch.equal(Y.s, Z.s)
    Z.q[:, 40] = -127
    assert torch.equal(Y.q, Z.q)
    check_status()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_smooth_activations_of_nan_and_infinities(act, dt):
    """x Phi(x), x sigmoid(z): +inf times 1 is +inf, -inf times 0 and a NaN are NaN."""
    y = _forward(act, [NAN, INF, -INF], dt)
    assert torch.isnan(y[:, 0]).all() and (y[:, 1] == INF).all() and torch.isnan(y[:, 2]).all()
    assert torch.isfinite(y[:, 3:]).all()
    # the largest finite values stay finite: x for positive, 0 for negative ones
    big = torch.finfo(torch.float32).max
    y = _forward(act, [big, -big])
    assert (y[:, 0] == big).all() and (y[:, 1] == 0).all()
    check_status()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu"])
def test_infinity_makes_an_infinite_scale(act):
    """An overflow to +inf shows in the INT8 output as it does without an activation: the block's scale is infinite."""
    Y = _forward(act, [1.0, INF], None)
    assert (Y.s[:, 0] == INF).all() and torch.isfinite(Y.s[:, 1]).all()
    check_status()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu"])
def test_gradient_at_a_block_with_an_infinite_scale(act):
    """A pre-activation that overflowed leaves a block with an infinite scale, whose codes 0 stand for 0 times infinity: the
    derivative there is NaN (of ReLU 0, as for every value that is not above 0), not that of an ordinary 0. Blocks with
    finite scales keep their gradients."""
    P = jf.QTensor(torch.zeros(32, 64, dtype=torch.int8, device="cuda"), torch.tensor([[INF, 1.0]], device="cuda"))
    P.q[5, 7] = -127
    eye = jf.QTensor(torch.eye(64, dtype=torch.int8, device="cuda"), torch.ones(2, 2, device="cuda"))
    dY = jf.QTensor(torch.ones(32, 64, dtype=torch.int8, device="cuda"), torch.ones(1, 2, device="cuda"))
    z = jf.linear_dgrad_epilogue(dY, eye, P, act, out_dtype=torch.float32)
    zero = z[:, :32].flatten()[P.q[:, :32].flatten() == 0]
    assert (zero == 0).all() if act == "relu" else torch.isnan(zero).all()
    assert (z[:, 32:] == (0.0 if act == "relu" else 0.5)).all()
    check_status()
