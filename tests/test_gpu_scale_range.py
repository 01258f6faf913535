"""Block-scaled products at scale products far from 1: c = fp32(sA sB) from subnormal to near the largest fp32.
Every entry point forms sum over the contraction blocks of c P in fp32, so a finite c P gives a finite term and a
block whose partial P is 0 gives 0, whatever c."""
import pytest
import torch

import int8_fully_quantized_b200 as jf

from gpu_common import GEMM_RTOL, check_status

pytestmark = pytest.mark.gpu

OPS = ["fwd", "dgrad", "wgrad", "fwd_gelu", "fwd_epilogue", "dgrad_epilogue"]


def _product(op, aq, a_s, bq, b_s):
    """The fp32 product of A [rows, K] and B [cols, K] (codes, and scales [rows / 32, K / 32]) through one entry point;
    fwd_gelu has no dense output: the value of its INT8 pre-activation."""
    t = lambda x: x.t().contiguous()
    A, Bt = jf.QTensor(aq, a_s), jf.QTensor(bq, b_s)
    y = torch.empty(aq.shape[0], bq.shape[0], device="cuda")
    if op == "fwd":
        jf.jf_linear_fwd(A, Bt, None, y)
    elif op == "dgrad":
        jf.jf_linear_dgrad(A, jf.QTensor(t(bq), t(b_s)), None, y)
    elif op == "wgrad":
        jf.jf_linear_wgrad(jf.QTensor(t(aq), t(a_s)), jf.QTensor(t(bq), t(b_s)), None, y)
    elif op == "fwd_epilogue":
        jf.jf_linear_fwd_epilogue(A, Bt, y=y)
    elif op == "dgrad_epilogue":
        jf.jf_linear_dgrad_epilogue(A, jf.QTensor(t(bq), t(b_s)), dx=y)
    else:
        Y, P = jf.empty_qtensor(*y.shape), jf.empty_qtensor(*y.shape)
        jf.jf_linear_fwd_gelu(A, Bt, Y, P)
        return P
    return y


def _partials(aq, a_s, bq, b_s):
    """[K / 32, rows, cols] in fp64: c of each block with its one fp32 rounding, and the exact partial P."""
    rows, K = aq.shape
    a = aq.double().reshape(rows, K // 32, 32).transpose(0, 1)
    b = bq.double().reshape(-1, K // 32, 32).transpose(0, 1)
    c = (a_s[:, None, :] * b_s[None, :, :]).double()          # fp32 product, widened
    c = c.permute(2, 0, 1).repeat_interleave(32, 1).repeat_interleave(32, 2)
    return c, a @ b.transpose(1, 2)


# contraction blocks: one; a tile's odd end; two windows of 32 blocks and an odd end; four CTAs' shares of a split one
@pytest.mark.parametrize("rows,cols,K", [(32, 32, 32), (96, 160, 96), (160, 96, 2080), (32, 64, 4096)])
@pytest.mark.parametrize("op", OPS)
def test_scale_products_over_the_range_of_fp32(op, rows, cols, K):
    """Codes of -1, 0 and 1 in single contraction blocks, c from 2^-149 to 2^122: each output is one block's c P, exact in
    fp32 (a sum with zeros, |P| <= 32), and 0 where the partials are. INT8 outputs: within half a code."""
    g = torch.Generator(device="cuda").manual_seed(rows + 3 * cols + 5 * K)
    kb = K // 32
    for n, e in enumerate((-149, -130, -60, 0, 104, 105, 106, 114, 122)):
        at = (7 * n) % kb
        aq = torch.zeros(rows, K, dtype=torch.int8, device="cuda")
        bq = torch.randint(-1, 2, (cols, K), generator=g, device="cuda", dtype=torch.int8)
        aq[:, 32 * at:32 * at + 32] = torch.randint(-1, 2, (rows, 32), generator=g, device="cuda", dtype=torch.int8)
        aq[1] = 0                                              # P = 0 in every block
        a_s = torch.full((rows // 32, kb), 2.0 ** (e // 2), device="cuda")
        b_s = torch.full((cols // 32, kb), 2.0 ** (e - e // 2), device="cuda")
        c, P = _partials(aq, a_s, bq, b_s)
        want = (c * P).sum(0)
        y = _product(op, aq, a_s, bq, b_s)
        if op == "fwd_gelu":
            s = y.s.repeat_interleave(32, 0).repeat_interleave(32, 1).double()
            assert torch.isfinite(y.s).all()
            # s = absmax / 127 rounded, half of 2^-149 below the normal numbers; then half a code
            assert ((y.q.double() * s - want).abs() <= s * 0.5 * (1 + 2.0 ** -20) + 127 * 2.0 ** -150).all(), e
        else:
            assert torch.equal(y.double(), want), e
    check_status()


@pytest.mark.parametrize("op", [o for o in OPS if o != "fwd_gelu"])
def test_mixed_scale_products(op):
    """Blocks of every magnitude in one contraction: some windows of 32 blocks hold large products and others none, with
    zero partials among them. The order of the fp32 sum is free: 1e-5 of the sum of magnitudes, plus half of the
    smallest subnormal for each of the 67 + 8 roundings that may fall there."""
    rows, cols, K = 96, 128, 67 * 32
    g = torch.Generator(device="cuda").manual_seed(3)
    aq = torch.randint(-127, 128, (rows, K), generator=g, device="cuda", dtype=torch.int8)
    bq = torch.randint(-127, 128, (cols, K), generator=g, device="cuda", dtype=torch.int8)
    e = torch.tensor([-40, 0, 20, 40, 53], device="cuda")
    a_s = torch.exp2(e[torch.randint(0, 5, (rows // 32, K // 32), generator=g, device="cuda")].float())
    b_s = torch.exp2(e[torch.randint(0, 5, (cols // 32, K // 32), generator=g, device="cuda")].float())
    a_s[0] = 2.0 ** -40                                        # a row block without large products
    a_s[1, :32], a_s[1, 32:] = 1.0, 2.0 ** 53                  # and one with them from its second window on
    aq[32:64, 32 * 40:] = 0                                    # whose partials are 0 after eight blocks
    c, P = _partials(aq, a_s, bq, b_s)
    y = _product(op, aq, a_s, bq, b_s).double()
    mag = (c * P.abs()).sum(0)
    assert torch.isfinite(y).all() and mag.max() > 2.0 ** 106
    assert ((y - (c * P).sum(0)).abs() <= GEMM_RTOL * mag + 75 * 2.0 ** -150).all()
    check_status()


@pytest.mark.parametrize("op", [o for o in OPS if o != "fwd_gelu"])
def test_infinite_scale_products(op):
    """A scale product past the largest fp32 is infinite and its block's terms are infinite, NaN where the partial is 0
    (infinity times 0); rows that do not meet it keep their values."""
    aq = torch.ones(64, 64, dtype=torch.int8, device="cuda")
    bq = torch.ones(32, 64, dtype=torch.int8, device="cuda")
    aq[3, :32] = 0
    a_s, b_s = torch.ones(2, 2, device="cuda"), torch.ones(1, 2, device="cuda")
    a_s[0, 0], b_s[0, 0] = 2.0 ** 100, 2.0 ** 30
    a_s[1, 0] = 2.0 ** -30
    y = _product(op, aq, a_s, bq, b_s)
    assert torch.isnan(y[3]).all() and torch.isinf(y[:3]).all() and torch.isinf(y[4:32]).all()
    assert (y[32:] == 64).all()
    check_status()
