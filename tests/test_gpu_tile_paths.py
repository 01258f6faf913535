"""A linear product is computed by one of several instances, chosen by the number of output tiles and the length of the
contraction. What they compute per output block is the same arithmetic in the same order, so a block has the same bits
in a large call and in a small one that holds only its rows (or columns)."""
import pytest
import torch

import int8_fully_quantized_b200 as jf

import block_ref as B
from gpu_common import check_status

pytestmark = pytest.mark.gpu


def _qt(g, rows, cols, std=1.0):
    return jf.QTensor(*B.quantize(torch.randn(rows, cols, generator=g, device="cuda") * std))


def _rows(t, n):
    return jf.QTensor(t.q[:n].contiguous(), t.s[:n // 32].contiguous())


def _cols(t, n):
    return jf.QTensor(t.q[:, :n].contiguous(), t.s[:, :n // 32].contiguous())


# contractions: shorter and longer than the rule's border, one that is no whole stage, and a long one
@pytest.mark.parametrize("K", [32, 96, 128, 160, 1024, 1056])
def test_large_and_small_calls_agree(K):
    g = torch.Generator(device="cuda").manual_seed(K)
    M, N, m = 2080, 2080, 160                                   # 289 tiles and 34 of them
    X, W, WT, XT = _qt(g, M, K), _qt(g, N, K, 0.05), _qt(g, K, N, 0.05), _qt(g, K, M)
    Xs, XTs = _rows(X, m), _cols(XT, m)

    def outputs(rows):
        return jf.empty_qtensor(rows, N), torch.empty(rows, N, device="cuda"), jf.empty_qtensor(rows, N)

    def same(big, small):
        for a, b in zip(big, small):
            if isinstance(a, jf.QTensor):
                assert torch.equal(a.q[:m], b.q) and torch.equal(a.s[:m // 32], b.s)
            else:
                assert torch.equal(a[:m], b)

    calls = [
        lambda x, xt, o: jf.jf_linear_fwd(x, W, o[0], o[1]),
        lambda x, xt, o: jf.jf_linear_fwd(x, W, None, o[1]),
        lambda x, xt, o: jf.jf_linear_dgrad(x, WT, o[0], o[1]),
        lambda x, xt, o: jf.jf_linear_wgrad(xt, WT, o[0], o[1]),
        lambda x, xt, o: jf.jf_linear_fwd_gelu(x, W, o[0], o[2]),
    ]
    for i, call in enumerate(calls):
        big, small = outputs(M), outputs(m)
        call(X, XT, big)
        call(Xs, XTs, small)
        used = [(0, 1), (1,), (0, 1), (0, 1), (0, 2)][i]
        same([big[k] for k in used], [small[k] for k in used])
        if i == 0:
            q, s = B.quantize(big[1])
            assert torch.equal(q, big[0].q) and torch.equal(s, big[0].s)
    check_status()


@pytest.mark.parametrize("K", [0, 32, 128, 160])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_epilogues_of_many_tiles(K, act):
    """Bias, activation and residual over several tiles a CTA (an empty contraction among them), forward and input
    gradient, against the 64-bit form."""
    g = torch.Generator(device="cuda").manual_seed(K + 1)
    M, N = 2080, 2080
    X, W, WT = (jf.empty_qtensor(M, 0), jf.empty_qtensor(N, 0), jf.empty_qtensor(0, N)) if K == 0 else \
        (_qt(g, M, K), _qt(g, N, K, 0.05), _qt(g, K, N, 0.05))
    xv, wv, tv = (torch.zeros(M, 1, device="cuda", dtype=torch.float64), torch.zeros(N, 1, device="cuda", dtype=torch.float64),
                  torch.zeros(1, N, device="cuda", dtype=torch.float64)) if K == 0 else (B.value(*X), B.value(*W), B.value(*WT))
    bias, r, P = torch.randn(N, generator=g, device="cuda"), torch.randn(M, N, generator=g, device="cuda"), _qt(g, M, N)
    p = xv @ wv.t() + bias.double()
    z = B.act(p, act) + r.double()
    y, pre = jf.linear_fwd_epilogue(X, W, bias, act, r, want_pre=True, out_dtype=torch.float32)
    # as in the epilogues' own tests: 1.13 (1e-5 of the sum of magnitudes) and 2^-18 of what is added
    tol = 1.13e-5 * (xv.abs() @ wv.abs().t()) + 2.0 ** -18 * (p.abs() + z.abs() + r.double().abs())
    assert ((y.double() - z).abs() <= tol).all()
    q, s = B.quantize(p)
    assert (pre.s - s).abs().max() <= 1e-5 * s.max() and (pre.q.int() - q.int()).abs().max() <= 1
    Y = jf.linear_fwd_epilogue(X, W, bias, act, r)
    q, s = B.quantize(y)
    assert torch.equal(q, Y.q) and torch.equal(s, Y.s)
    d = jf.linear_dgrad_epilogue(X, WT, P, act, r, out_dtype=torch.float32)
    dz = (xv @ tv) * B.act_grad(B.value(*P), act) + r.double()
    tol = 1.13e-5 * (xv.abs() @ tv.abs()) + 2.0 ** -18 * ((xv @ tv).abs() + dz.abs() + r.double().abs())
    assert ((d.double() - dz).abs() <= tol).all()
    check_status()
