"""GPU tests of the linear layer's epilogues (bias, activation, residual; activation gradient) and of the
bias gradient against 64-bit plain forms.

Tolerances, fixed before the first run. The product obeys the GEMM tolerance of gpu_common (1e-5 of its
condition scale mag = sum of |terms|). Bias, residual and activation add a few fp32 roundings of values no larger
than |p| + |r| + |z|; activations and their derivatives (both bounded by 1.13) are within 2^-18 relative of
their formula in fp32 (the erfc fit's 5e-6 bound dominates), and |act'| <= 1.13 carries the product's error on.
So |z - z64| <= 1.13 (1e-5 mag) + 2^-18 (|p| + |r| + |z|), plus half a step of the output type. INT8 outputs: the
re-quantization rule of gpu_common."""
import numpy as np
import pytest
import torch

import int8_fully_quantized_b200 as jf

import block_ref as B
from gpu_common import GEMM_RTOL, assert_requant_close, check_status, host

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _qt(g, rows, cols, std=1.0):
    x = torch.randn(rows, cols, generator=g, device="cuda") * std
    if cols > 64:
        x[:, 5::97] *= 20.0
    return jf.QTensor(*B.quantize(x))


def _residual(g, kind, rows, cols):
    if kind == "none":
        return None, 0.0
    x = torch.randn(rows, cols, generator=g, device="cuda")
    if kind == "i8":
        q = jf.QTensor(*B.quantize(x))
        return q, B.value(*q)
    x = x.to({"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[kind])
    return x, x.double()


def _close(z, z64, tol, what):
    d = (z.double() - z64).abs() - (tol + B.HALF_STEP[z.dtype] * z64.abs() * (1 + 2.0 ** -7) + B.TINY[z.dtype])
    assert d.max().item() <= 0, f"{what}: {d.max().item():.3e} beyond the tolerance"


def _codes_close(t, z64, what):
    q, s = B.quantize(z64)
    assert_requant_close(host(t.q), host(t.s), q.cpu().numpy(), s.cpu().numpy(), what)


SHAPES = [(32, 32, 32), (32, 64, 96), (96, 32, 160), (160, 352, 32), (352, 544, 1056), (224, 1024, 64), (1024, 160, 512)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act,res", [("none", "none"), ("gelu", "i8"), ("gelu_tanh", "fp32"), ("silu", "bf16"), ("relu", "fp16")])
def test_forward(M, N, K, act, res):
    g = _gen(M + 3 * N + 7 * K)
    X, W = _qt(g, M, K), _qt(g, N, K, 0.05)
    bias = torch.randn(N, generator=g, device="cuda")
    r, r64 = _residual(g, res, M, N)
    xv, wv = B.value(*X), B.value(*W)
    p = xv @ wv.t() + bias.double()
    mag = xv.abs() @ wv.abs().t()
    z = B.act(p, act) + r64
    tol = 1.13 * GEMM_RTOL * mag + 2.0 ** -18 * (p.abs() + z.abs() + (r64.abs() if res != "none" else 0.0))
    Y, P = jf.linear_fwd_epilogue(X, W, bias, act, r, want_pre=True)
    _codes_close(Y, z, "Y")
    _codes_close(P, p, "P")
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        _close(jf.linear_fwd_epilogue(X, W, bias, act, r, out_dtype=dt), z, tol, f"dense {dt}")
    # without a bias; and both outputs of one call are the same values
    y = torch.empty(M, N, device="cuda")
    Y2 = jf.empty_qtensor(M, N)
    jf.jf_linear_fwd_epilogue(X, W, Y2, y, None, act, r)
    _close(y, B.act(p - bias.double(), act) + r64, tol + 2.0 ** -18 * bias.abs().double(), "no bias")
    q, s = B.quantize(y)
    assert torch.equal(q, Y2.q) and torch.equal(s, Y2.s)
    check_status()


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("act,res", [("none", "bf16"), ("gelu", "none"), ("gelu_tanh", "i8"), ("silu", "fp32"), ("relu", "fp16")])
def test_input_gradient(M, K, N, act, res):
    g = _gen(M + 5 * N + 11 * K)
    dY, W, P = _qt(g, M, N, 1e-2), _qt(g, N, K, 0.05), _qt(g, M, K, 1.5)
    P.q[0, :32] = torch.arange(-128, -96, device="cuda", dtype=torch.int8)     # -128 is accepted on input
    r, r64 = _residual(g, res, M, K)
    dv, wv, pv = B.value(*dY), B.value(*W), B.value(*P)
    gr = B.act_grad(pv, act)
    z = (dv @ wv) * gr + r64
    tol = 1.13 * GEMM_RTOL * (dv.abs() @ wv.abs()) + 2.0 ** -18 * ((dv @ wv).abs() + z.abs() + (r64.abs() if res != "none" else 0.0))
    _codes_close(jf.linear_dgrad_epilogue(dY, W, P, act, r), z, "dX")
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        _close(jf.linear_dgrad_epilogue(dY, W, P, act, r, out_dtype=dt), z, tol, f"dense {dt}")
    check_status()


# few output tiles and a long contraction, which clusters of CTAs share: 8 parts; 8 of which two are empty; 8 with a
# last one of a single block; 4 of which one is empty; 4; 2 of one stage each
@pytest.mark.parametrize("M,N,K", [(32, 64, 4096), (160, 352, 2080), (32, 32, 3616), (352, 544, 1056), (128, 4096, 544), (1024, 1024, 256)])
def test_shared_contraction(M, N, K):
    """Forward and input gradient as above, the same bits at every call, on two streams at once and replayed."""
    g = _gen(M + N + K)
    X, W, dY, WT = _qt(g, M, K), _qt(g, N, K, 0.05), _qt(g, M, K, 1e-2), _qt(g, K, N, 0.05)
    P = _qt(g, M, N, 1.5)
    bias = torch.randn(N, generator=g, device="cuda")
    r = torch.randn(M, N, generator=g, device="cuda")
    xv, wv, dv, tv = B.value(*X), B.value(*W), B.value(*dY), B.value(*WT)
    p = xv @ wv.t() + bias.double()
    z = B.act(p, "gelu") + r.double()
    tol = 1.13 * GEMM_RTOL * (xv.abs() @ wv.abs().t()) + 2.0 ** -18 * (p.abs() + z.abs() + r.double().abs())
    y = jf.linear_fwd_epilogue(X, W, bias, "gelu", r, out_dtype=torch.float32)
    _close(y, z, tol, "dense")
    Y, pre = jf.linear_fwd_epilogue(X, W, bias, "gelu", r, want_pre=True)
    q, s = B.quantize(y)
    assert torch.equal(q, Y.q) and torch.equal(s, Y.s)
    _codes_close(pre, p, "P")
    d = jf.linear_dgrad_epilogue(dY, WT, P, "gelu", r, out_dtype=torch.float32)
    dz = (dv @ tv) * B.act_grad(B.value(*P), "gelu") + r.double()
    _close(d, dz, 1.13 * GEMM_RTOL * (dv.abs() @ tv.abs()) + 2.0 ** -18 * ((dv @ tv).abs() + dz.abs() + r.double().abs()), "input gradient")
    side = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.empty_like(y) for _ in range(8)]
    torch.cuda.synchronize()
    for i, o in enumerate(ys):
        if i % 2:
            jf.jf_linear_dgrad_epilogue(dY, WT, dx=o, pre=P, act="gelu", residual=r, stream=side[i // 2 % 2])
        else:
            jf.jf_linear_fwd_epilogue(X, W, y=o, bias=bias, act="gelu", residual=r, stream=side[i // 2 % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, d if i % 2 else y) for i, o in enumerate(ys))
    out, graph = torch.empty_like(y), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jf.jf_linear_fwd_epilogue(X, W, y=out, bias=bias, act="gelu", residual=r)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, y)
    check_status()


@pytest.mark.parametrize("act", B.ACTS)
def test_activation_gradient_against_differences(act):
    """dY = I in 32 x 32 blocks through W = I: Z = act'(P) itself, against central differences of the
    activation (h = 2^-10: h^2 / 6 |f'''| with |f'''| < 3, plus fp32's 2^-18)."""
    P = jf.QTensor(*B.quantize(torch.linspace(-8, 8, 32 * 32, device="cuda").reshape(32, 32) + 1e-3))
    eye = jf.QTensor(*B.quantize(torch.eye(32, device="cuda")))
    ones = jf.QTensor(*B.quantize(torch.ones(32, 32, device="cuda")))
    z = jf.linear_dgrad_epilogue(ones, eye, P, act, out_dtype=torch.float32).double()
    x, h = B.value(*P), 2.0 ** -10
    diff = (B.act(x + h, act) - B.act(x - h, act)) / (2 * h)
    smooth = (x.abs() > 2 * h) if act == "relu" else torch.ones_like(x, dtype=torch.bool)
    unit = 127 * (1 / 127)      # the value of a coded 1: 127 * fp32(1 / 127), within 2^-23 of 1, and squared
    tol = h * h / 2 + 2.0 ** -18 + 2.0 ** -21 * unit
    assert ((z - diff).abs()[smooth] <= tol).all()


def test_activations_over_their_whole_range():
    """act(bias) alone (an empty contraction): signed powers of two from the smallest to the largest normal
    numbers, where exponentials under- and overflow. Errors relative to max(|act|, |x| 2^-18): what is below
    that is what exp(-x) or erfc(x) rounded away."""
    e = torch.arange(-126, 127, device="cuda")
    x = torch.cat([torch.ldexp(torch.full_like(e, s, dtype=torch.float32), e) for s in (1.0, -1.0, 1.5, -1.5)])
    x = torch.cat([x, torch.zeros(32 - x.numel() % 32, device="cuda")])
    X, W = jf.empty_qtensor(32, 0), jf.empty_qtensor(x.numel(), 0)
    for act in B.ACTS:
        y = jf.linear_fwd_epilogue(X, W, x, act, out_dtype=torch.float32)
        assert torch.isfinite(y).all() and (y == y[0]).all()
        xd = x.double()
        ref = torch.where(xd.abs() > 1e30, xd.clamp(min=0) if act != "none" else xd, B.act(xd.clamp(-1e30, 1e30), act))
        if act == "gelu_tanh":   # x^3 of the reference overflows nothing, but its tail is below fp32
            ref = torch.nan_to_num(ref)
        assert ((y[0].double() - ref).abs() <= 2.0 ** -17 * torch.maximum(ref.abs(), xd.abs() * 2.0 ** -18) + 2.0 ** -126).all(), act


def test_empty_contraction_and_empty_outputs():
    g = _gen(1)
    X, W = jf.empty_qtensor(64, 0), jf.empty_qtensor(96, 0)
    bias = torch.randn(96, generator=g, device="cuda")
    r = torch.randn(64, 96, generator=g, device="cuda").to(torch.bfloat16)
    z = B.act(bias.double(), "silu") + r.double()
    _close(jf.linear_fwd_epilogue(X, W, bias, "silu", r, out_dtype=torch.float32), z, 2.0 ** -18 * (z.abs() + r.double().abs() + bias.abs().double()), "K = 0")
    _codes_close(jf.linear_fwd_epilogue(X, W, bias, "silu", r), z, "K = 0")
    zero = jf.linear_dgrad_epilogue(jf.empty_qtensor(64, 0), jf.empty_qtensor(0, 96))
    assert not host(zero.q).any() and not host(zero.s).any()
    for M, N in ((0, 64), (64, 0)):
        Y, P = jf.linear_fwd_epilogue(jf.empty_qtensor(M, 64), jf.empty_qtensor(N, 64), torch.zeros(N, device="cuda"), "gelu", want_pre=True)
        assert Y.q.shape == (M, N) and P.q.shape == (M, N)
        assert jf.linear_fwd_epilogue(jf.empty_qtensor(M, 64), jf.empty_qtensor(N, 64), out_dtype=torch.float16).shape == (M, N)
    check_status()


def _ieee_codes(x):
    """s = absmax / 127 and the codes RNE(RN(x / s)) in IEEE fp32 on the host; zero blocks get zeros."""
    M, N = x.shape
    b = x.cpu().reshape(M // 32, 32, N // 32, 32)
    s = b.abs().amax(dim=(1, 3)) / torch.tensor(127.0)
    sb = s[:, None, :, None]
    q = torch.where(sb == 0, torch.zeros_like(b), (b / torch.where(sb == 0, torch.ones_like(sb), sb)).clamp(-127, 127).round())
    return q.to(torch.int8).reshape(M, N), s


def _tie_dense(g, rows, cols):
    """Blocks whose values are (n + 1/2) s rounded, up to 3 units in the last place to either side, for scales from
    the smallest subnormals (where a block's codes may all be 0) to near the largest fp32."""
    nr, nc = rows // 32, cols // 32
    e = torch.linspace(-150, 119, nr * nc, device="cuda").reshape(nr, 1, nc, 1)
    s = ((torch.rand(nr, 1, nc, 1, generator=g, device="cuda") + 1) * torch.exp2(e)).to(torch.float32)
    s = torch.where(e < -140, torch.exp2(e.double()).to(torch.float32), s)
    top = (127.0 * s.double()).to(torch.float32)
    sc = (top.cpu() / torch.tensor(127.0)).cuda()
    n = torch.randint(-126, 126, (nr, 32, nc, 32), generator=g, device="cuda")
    x = ((n.double() + 0.5) * sc.double()).to(torch.float32)
    x = (x.view(torch.int32) + torch.randint(-3, 4, x.shape, generator=g, device="cuda", dtype=torch.int32) * (x.abs() > 1e-44)).view(torch.float32)
    x = torch.minimum(torch.maximum(x, -top), top)
    x[:, 0, :, 0] = top[:, 0, :, 0]
    return x.reshape(rows, cols)


def test_codes_next_to_rounding_ties():
    """The codes of the epilogue and of the QKV gradient are those of the IEEE quotient, for values next to rounding
    ties and scales over the whole range: the residual alone (an empty contraction, no activation) and values'
    gradients pass through unchanged before they are quantized."""
    g = _gen(21)
    x = _tie_dense(g, 512, 1088)
    assert torch.isfinite(x).all()
    q, s = _ieee_codes(x)
    Y = jf.linear_fwd_epilogue(jf.empty_qtensor(512, 0), jf.empty_qtensor(1088, 0), residual=x)
    assert torch.equal(Y.s.cpu(), s) and torch.equal(Y.q.cpu(), q)
    for d in (32, 64, 96, 128, 256):
        h = 1088 // d - (1088 // d) % 2
        c = x[:, :h * d].contiguous()
        q, s = _ieee_codes(c)
        a = jf.QKVRope(1, 512, 0, h // 2, d)
        half = h // 2 * d
        dx, _, _ = jf.qkv_rope_bwd(jf.empty_qtensor(512, h * d), a, None, c[:, :half].reshape(1, 512, h // 2, d), c[:, half:].reshape(1, 512, h // 2, d))
        assert torch.equal(dx.s.cpu(), s) and torch.equal(dx.q.cpu(), q), d
    check_status()


def test_codes_of_infinities_and_nan():
    """A NaN leaves its block's scale and the other codes as they are and gets -127; an infinity makes the scale
    infinite, the finite codes 0 and its own -127."""
    x = torch.randn(64, 96, generator=_gen(22), device="cuda")
    y = x.clone()
    y[3, 5], y[40, 70] = float("nan"), float("inf")
    W = (jf.empty_qtensor(64, 0), jf.empty_qtensor(96, 0))
    A, Bq = jf.linear_fwd_epilogue(*W, residual=x), jf.linear_fwd_epilogue(*W, residual=y)
    clean = x.clone()
    clean[3, 5] = 0.0
    q, s = _ieee_codes(clean)
    q[3, 5] = -127
    q[32:, 64:] = 0
    q[40, 70] = -127
    s[1, 2] = float("inf")
    assert torch.equal(Bq.q.cpu(), q) and torch.equal(Bq.s.cpu(), s)
    assert torch.equal(A.q.cpu(), _ieee_codes(x)[0])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_strided_rows_in_place_and_guards(dt):
    """The residual stream as columns of a wider buffer, updated in place: the other columns and the rows
    around it keep their bytes."""
    g = _gen(2)
    M, N, K = 160, 224, 96
    X, W = _qt(g, M, K), _qt(g, N, K, 0.05)
    bias = torch.randn(N, generator=g, device="cuda")
    wide = torch.randn(M + 2, N + 64, generator=g, device="cuda").to(dt)
    before = wide.clone()
    view = wide[1:M + 1, 32:32 + N]
    want = jf.linear_fwd_epilogue(X, W, bias, "gelu", view.contiguous(), out_dtype=dt)
    jf.jf_linear_fwd_epilogue(X, W, y=view, bias=bias, act="gelu", residual=view)
    assert torch.equal(view, want)
    view.copy_(before[1:M + 1, 32:32 + N])
    assert torch.equal(wide, before)
    with pytest.raises(jf.JetfireError, match="misaligned"):
        jf.jf_linear_fwd_epilogue(X, W, y=wide[1:M + 1, 33:33 + N])
    with pytest.raises(jf.JetfireError, match="overlaps"):
        jf.jf_linear_fwd_epilogue(X, W, y=wide[1:M + 1, 32:32 + N], residual=wide[0:M, 32:32 + N])
    with pytest.raises(ValueError, match="device memory"):
        jf.linear_fwd_epilogue(jf.QTensor(X.q.cpu(), X.s.cpu()), jf.QTensor(W.q.cpu(), W.s.cpu()))
    with pytest.raises(ValueError, match="in one call"):
        jf.linear_fwd_epilogue(X, W, bias.cpu())


def test_side_stream_and_graph_replay():
    """A call on a side stream, and a captured one replayed on new inputs, equal the eager call."""
    g = _gen(3)
    X, W, P = _qt(g, 256, 128), _qt(g, 384, 128, 0.05), _qt(g, 256, 128)
    dY = _qt(g, 256, 384, 1e-2)
    bias = torch.randn(384, generator=g, device="cuda")
    want, pre = jf.linear_fwd_epilogue(X, W, bias, "gelu", want_pre=True)
    want_d, want_b = jf.linear_dgrad_epilogue(dY, W, P, "gelu"), jf.bias_grad(dY)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y, d, b = jf.linear_fwd_epilogue(X, W, bias, "gelu"), jf.linear_dgrad_epilogue(dY, W, P, "gelu"), jf.bias_grad(dY)
    side.synchronize()
    z = jf.linear_fwd_epilogue(X, W, bias, "gelu", stream=side)
    side.synchronize()
    for a, c in ((y, want), (d, want_d), (z, want)):
        assert torch.equal(a.q, c.q) and torch.equal(a.s, c.s)
    assert torch.equal(b, want_b)
    Y, DX, DB = jf.empty_qtensor(256, 384), jf.empty_qtensor(256, 128), torch.empty(384, device="cuda")
    Xs = jf.QTensor(X.q.clone(), X.s.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jf.jf_linear_fwd_epilogue(Xs, W, Y, bias=bias, act="gelu")
        jf.jf_linear_dgrad_epilogue(dY, W, DX, pre=P, act="gelu")
        jf.jf_bias_grad(dY, DB)
    X2 = _qt(g, 256, 128)
    for src in (X, X2):
        Xs.q.copy_(src.q)
        Xs.s.copy_(src.s)
        graph.replay()
        ref = jf.linear_fwd_epilogue(src, W, bias, "gelu")
        assert torch.equal(Y.q, ref.q) and torch.equal(Y.s, ref.s)
        assert torch.equal(DX.q, want_d.q) and torch.equal(DB, want_b)
    check_status()


@pytest.mark.parametrize("M,N", [(32, 32), (32, 96), (64, 160), (288, 1056), (2080, 96), (8192, 512), (65536, 32)])
def test_bias_grad(M, N):
    """Integer sums per 8 rows are exact; what is left are M / 8 products and sums in fp32 in some order:
    within (M / 8 + 20) 2^-24 of the sum of magnitudes at worst; sums of 9 or more blocks per lane do not occur
    below M = 16384, so 2^-18 of it covers every case here."""
    g = _gen(M + N)
    dY = _qt(g, M, N, 1e-3)
    dY.q[0, :] = -128
    v = B.value(*dY)
    db = jf.bias_grad(dY)
    assert ((db.double() - v.sum(0)).abs() <= 2.0 ** -18 * v.abs().sum(0)).all()
    assert torch.equal(db, jf.bias_grad(dY))                         # the same bits every time


def test_bias_grad_empty_and_past_32_bits():
    assert not host(jf.bias_grad(jf.empty_qtensor(0, 96))).any()
    assert jf.bias_grad(jf.empty_qtensor(64, 0)).numel() == 0
    # 2^31 + 2^20 codes: offsets past 32 bits
    M, N = 65568, 32768
    q = torch.randint(-127, 128, (M, N), dtype=torch.int8, device="cuda", generator=_gen(5))
    s = torch.full((M // 32, N // 32), 2.0 ** -10, device="cuda")
    db = jf.bias_grad(jf.QTensor(q, s))
    for c0 in (0, 16384, N - 256):
        want = q[:, c0:c0 + 256].sum(0, dtype=torch.int64).double() * 2.0 ** -10
        # equal scales and sums below 2^24: exact in fp32
        assert torch.equal(db[c0:c0 + 256].double(), want)
    check_status()
