"""Refusals of the transformer-block operators (linear epilogues, bias gradient, rotary tables, QKV norm and
rotation) and the host logic of their binding; nothing here needs a GPU: every call fails its checks before
it touches a device."""
import ctypes
import math

import pytest
import torch

import int8_fully_quantized_b200 as jf
from int8_fully_quantized_b200 import build_lib

import block_ref as B

NULL, SHAPE, ALIGN, DTYPE, ALIAS, DEVICE, WORKSPACE, ARG = -1, -2, -3, -4, -5, -8, -9, -10


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return jf.load_library()


def at(n):
    """A fake, 16-byte aligned device address, far from the other numbers' (never dereferenced)."""
    return n << 32


def cq(n, rows, cols):
    return jf._CQ(at(n), at(n) + (1 << 31), rows, cols)


def oq(n, rows, cols):
    return jf._Q(at(n), at(n) + (1 << 31), rows, cols)


def mat(n, ld, dt=1):
    return jf._Matrix(at(n), dt, ld)


NOCQ, NOQ, NOM = jf._CQ(None, None, 0, 0), jf._Q(None, None, 0, 0), jf._Matrix(None, 0, 0)


def _fwd(lib, X=cq(1, 64, 96), W=cq(2, 32, 96), bias=at(3), act=2, Rq=NOCQ, R=NOM, Y=oq(5, 64, 32), y=NOM, P=NOQ):
    return lib.jf_linear_fwd_epilogue(X, W, bias, act, Rq, R, Y, y, P, None)


def _bwd(lib, dY=cq(1, 64, 96), W=cq(2, 96, 32), P=cq(3, 64, 32), act=2, Rq=NOCQ, R=NOM, Y=oq(5, 64, 32), y=NOM):
    return lib.jf_linear_dgrad_epilogue(dY, W, P, act, Rq, R, Y, y, None)


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: checked without a device only")


@no_gpu
def test_linear_epilogue_valid_calls_stop_only_at_the_device(lib):
    assert _fwd(lib) == DEVICE
    assert _fwd(lib, bias=None, act=0, Y=NOQ, y=mat(6, 32)) == DEVICE
    assert _fwd(lib, P=oq(7, 64, 32), R=mat(8, 40, 0)) == DEVICE
    assert _fwd(lib, Rq=cq(8, 64, 32)) == DEVICE
    assert _fwd(lib, Y=NOQ, y=mat(6, 32), R=mat(6, 32)) == DEVICE            # the residual updated in place
    assert _fwd(lib, X=jf._CQ(None, None, 64, 0), W=jf._CQ(None, None, 32, 0)) == DEVICE   # empty contraction
    assert _bwd(lib) == DEVICE
    assert _bwd(lib, act=0, P=NOCQ) == DEVICE
    assert lib.jf_bias_grad(cq(1, 64, 96), at(2), None) == DEVICE


def test_linear_epilogue_refusals(lib):
    assert _fwd(lib, act=5) == ARG and _fwd(lib, act=-1) == ARG
    assert _fwd(lib, Rq=cq(8, 64, 32), R=mat(9, 32)) == ARG                  # two residuals
    assert _fwd(lib, Y=NOQ) == NULL                                          # no output
    assert _fwd(lib, X=cq(1, 64, 64)) == SHAPE
    assert _fwd(lib, Y=oq(5, 64, 64)) == SHAPE and _fwd(lib, P=oq(7, 32, 32)) == SHAPE
    assert _fwd(lib, Rq=cq(8, 32, 32)) == SHAPE
    assert _fwd(lib, R=mat(9, 24)) == SHAPE and _fwd(lib, y=mat(9, 31)) == SHAPE    # pitch below the width
    assert _fwd(lib, R=mat(9, 33)) == ALIGN                                  # pitch not a multiple of 16 bytes
    assert _fwd(lib, R=jf._Matrix(at(9) + 8, 1, 32)) == ALIGN and _fwd(lib, bias=at(3) + 4) == ALIGN
    assert _fwd(lib, R=mat(9, 32, 3)) == DTYPE and _fwd(lib, y=mat(9, 32, -1)) == DTYPE
    # outputs over inputs and over each other; y over R but not the same view
    assert _fwd(lib, Y=oq(1, 64, 32)) == ALIAS and _fwd(lib, P=oq(5, 64, 32)) == ALIAS
    assert _fwd(lib, y=mat(5, 32)) == ALIAS and _fwd(lib, y=mat(3, 32)) == ALIAS
    assert _fwd(lib, y=mat(9, 32), R=mat(9, 40)) == ALIAS and _fwd(lib, y=mat(9, 32, 0), R=mat(9, 32, 1)) == ALIAS
    assert _fwd(lib, Y=oq(8, 64, 32), Rq=cq(8, 64, 32)) == ALIAS
    # empty outputs are no-ops, whatever else is missing
    assert _fwd(lib, X=jf._CQ(None, None, 0, 96), Y=jf._Q(None, None, 0, 32)) == 0
    assert _bwd(lib, P=NOCQ) == SHAPE and _bwd(lib, P=jf._CQ(None, None, 64, 32)) == NULL
    assert _bwd(lib, W=cq(2, 64, 32)) == SHAPE and _bwd(lib, act=9) == ARG
    assert _bwd(lib, Y=oq(3, 64, 32)) == ALIAS
    assert lib.jf_bias_grad(cq(1, 64, 96), None, None) == NULL
    assert lib.jf_bias_grad(cq(1, 64, 96), at(2) + 2, None) == ALIGN
    assert lib.jf_bias_grad(cq(1, 64, 96), at(1) + 64, None) == ALIAS
    assert lib.jf_bias_grad(cq(1, 64, 48), at(2), None) == SHAPE
    assert lib.jf_bias_grad(jf._CQ(None, None, 64, 0), None, None) == 0


def rope(batch=2, seq=20, hq=2, hkv=1, d=64, rot=64, layout=0, table=64, positions=None, gq=at(40), gk=at(41), eps=1e-6,
         cos=at(42), sin=at(43)):
    return jf._Rope(batch, seq, hq, hkv, d, rot, layout, cos, sin, table, positions, gq, gk, eps)


def heads(n, hs=64, ss=256, bs=20 * 256):
    return jf._Heads(at(n), bs, ss, hs)


def _qkv(lib, a, X=cq(1, 64, 256), q=heads(10), k=heads(11), v=heads(12), dt=1):
    return lib.jf_qkv_rope_fwd(X, ctypes.byref(a), q, k, v, dt, None)


def _qkv_bwd(lib, a, X=cq(1, 64, 256), q=heads(10), k=heads(11), v=heads(12), dt=1, dX=oq(20, 64, 256), dgq=at(30),
             dgk=at(31), ws=at(32), n=1 << 20):
    return lib.jf_qkv_rope_bwd(X, ctypes.byref(a), q, k, v, dt, dX, dgq, dgk, ws, n, None)


@no_gpu
def test_qkv_valid_calls_stop_only_at_the_device(lib):
    assert _qkv(lib, rope()) == DEVICE and _qkv_bwd(lib, rope()) == DEVICE
    assert _qkv(lib, rope(rot=0, cos=None, sin=None, table=0)) == DEVICE
    assert _qkv(lib, rope(table=8, positions=at(44))) == DEVICE
    assert _qkv(lib, rope(hkv=0, hq=4), k=jf._Heads(None, 0, 0, 0), v=jf._Heads(None, 0, 0, 0)) == DEVICE
    # views of one buffer; strides of dimensions of one element do not count
    assert _qkv(lib, rope(), q=jf._Heads(at(10), 20 * 256, 256, 64), k=jf._Heads(at(10) + 256, 20 * 256, 256, 7),
                v=jf._Heads(at(10) + 384, 20 * 256, 256, -3)) == DEVICE
    assert _qkv_bwd(lib, rope(), q=jf._Heads(at(10), 0, 0, 0)) == DEVICE     # a broadcast gradient
    # without a norm the codes are not read
    assert _qkv_bwd(lib, rope(gq=None, gk=None), X=jf._CQ(None, None, 64, 256), dgq=None, dgk=None, ws=None, n=0) == DEVICE


def test_qkv_refusals(lib):
    for bad in (dict(d=48), dict(d=0), dict(d=288), dict(rot=8), dict(rot=72), dict(rot=80), dict(batch=-1), dict(seq=40),
                dict(hq=-1), dict(hq=3), dict(table=19), dict(table=-1)):
        assert _qkv(lib, rope(**bad)) == SHAPE, bad
        assert _qkv_bwd(lib, rope(**bad)) == SHAPE, bad
    for bad in (dict(layout=2), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan)):
        assert _qkv(lib, rope(**bad)) == ARG, bad
    assert _qkv(lib, rope(), dt=3) == DTYPE
    assert _qkv(lib, rope(cos=None)) == NULL and _qkv(lib, rope(), q=jf._Heads(None, 0, 0, 0)) == NULL
    assert lib.jf_qkv_rope_fwd(cq(1, 64, 256), None, heads(10), heads(11), heads(12), 1, None) == NULL
    for bad in (dict(gq=at(40) + 4), dict(cos=at(42) + 8), dict(positions=at(44) + 4)):
        assert _qkv(lib, rope(**bad)) == ALIGN, bad
    assert _qkv(lib, rope(), q=heads(10, ss=260)) == ALIGN and _qkv(lib, rope(), v=jf._Heads(at(12) + 8, 5120, 256, 64)) == ALIGN
    # an output whose elements share places: heads on top of each other, tokens too close, broadcast
    assert _qkv(lib, rope(), q=heads(10, hs=32)) == SHAPE and _qkv(lib, rope(), q=heads(10, ss=64)) == SHAPE
    assert _qkv(lib, rope(), q=heads(10, bs=0)) == SHAPE and _qkv(lib, rope(), q=heads(10, ss=-256)) == SHAPE
    assert _qkv(lib, rope(), q=heads(1)) == ALIAS and _qkv(lib, rope(positions=at(12))) == ALIAS
    # backward: shapes, workspace, weight gradients without weights
    assert _qkv_bwd(lib, rope(), dX=oq(20, 64, 192)) == SHAPE
    need = lib.jf_qkv_rope_bwd_workspace_bytes(64, ctypes.byref(rope()))
    assert need == 2 * 4 * 2 * 64 * 4                                          # strips x heads CTAs, two kinds
    assert lib.jf_qkv_rope_bwd_workspace_bytes(1 << 20, ctypes.byref(rope())) == 296 * 2 * 64 * 4
    assert lib.jf_qkv_rope_bwd_workspace_bytes(33, ctypes.byref(rope())) == -1
    assert lib.jf_qkv_rope_bwd_workspace_bytes(64, ctypes.byref(rope(d=48))) == -1
    assert _qkv_bwd(lib, rope(), ws=None) == WORKSPACE and _qkv_bwd(lib, rope(), n=need - 1) == WORKSPACE
    assert _qkv_bwd(lib, rope(), ws=at(32) + 8) == WORKSPACE
    assert _qkv_bwd(lib, rope(gq=None)) == NULL
    assert _qkv_bwd(lib, rope(), dX=oq(10, 64, 256)) == ALIAS and _qkv_bwd(lib, rope(), ws=at(20)) == ALIAS
    assert _qkv_bwd(lib, rope(), dgk=at(30) + 128) == ALIAS
    assert _qkv(lib, rope(batch=0)) == 0


def test_strides_past_any_address_space(lib):
    """Strides whose products would overflow 64 bits are refused instead of wrapping into a small extent."""
    assert _fwd(lib, y=mat(6, 1 << 58)) == SHAPE and _fwd(lib, R=mat(6, 1 << 58), y=NOM) == SHAPE
    for bad in (dict(hs=1 << 58), dict(ss=1 << 58), dict(bs=1 << 58), dict(bs=1 << 62)):
        assert _qkv(lib, rope(), q=heads(10, **bad)) == SHAPE, bad
        assert _qkv_bwd(lib, rope(), v=heads(12, **bad) if "hs" not in bad else heads(12, ss=1 << 59)) == SHAPE, bad


def test_rope_table_refusals(lib):
    f = (ctypes.c_double * 129)()
    assert lib.jf_rope_table(f, 0, 1.0, 4, at(1), at(2), None) == SHAPE
    assert lib.jf_rope_table(f, 129, 1.0, 4, at(1), at(2), None) == SHAPE
    assert lib.jf_rope_table(f, 8, 1.0, -1, at(1), at(2), None) == SHAPE
    assert lib.jf_rope_table(f, 8, 1.0, 4, None, at(2), None) == NULL
    assert lib.jf_rope_table(f, 8, 1.0, 4, at(1) + 4, at(2), None) == ALIGN
    assert lib.jf_rope_table(f, 8, 1.0, 4, at(1), at(1) + 64, None) == ALIAS
    assert lib.jf_rope_table(None, 8, 1.0, 0, None, None, None) == 0


def test_rope_frequencies():
    f, m = jf.rope_frequencies(8)
    assert m == 1.0 and f == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-14)
    assert jf.rope_frequencies(8, scaling="linear", factor=4.0)[0] == pytest.approx([x / 4 for x in f], rel=1e-14)
    n, _ = jf.rope_frequencies(64, scaling="ntk", factor=8.0)
    p, _ = jf.rope_frequencies(64)
    assert n[0] == 1.0 and n[-1] == pytest.approx(p[-1] / 8.0, rel=1e-12)      # fastest kept, slowest divided
    y, m = jf.rope_frequencies(64, scaling="yarn", factor=8.0, original_length=2048)
    assert m == pytest.approx(0.1 * math.log(8.0) + 1.0, rel=1e-14)
    turns = [2048 * x / (2 * math.pi) for x in p]
    for j in range(32):
        if turns[j] > 33 * 1.5:
            assert y[j] == p[j]
        if turns[j] < 1 / 1.5:
            assert y[j] == pytest.approx(p[j] / 8, rel=1e-14)
        assert p[j] / 8 * (1 - 1e-12) <= y[j] <= p[j]
    for bad in (dict(rot_dim=7), dict(rot_dim=8, scaling="other"), dict(rot_dim=8, scaling="linear", factor=0.0),
                dict(rot_dim=8, scaling="yarn", factor=2.0), dict(rot_dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            jf.rope_frequencies(**bad)


def test_binding_refuses_what_the_abi_cannot_see(lib):
    q = lambda r, c: jf.QTensor(torch.zeros(r, c, dtype=torch.int8), torch.zeros(r // 32, c // 32))
    X, W = q(64, 96), q(32, 96)
    with pytest.raises(ValueError, match="activation"):
        jf.linear_fwd_epilogue(X, W, act="swish")
    with pytest.raises(ValueError, match="bias"):
        jf.linear_fwd_epilogue(X, W, bias=torch.zeros(64))
    with pytest.raises(ValueError, match="bias"):
        jf.linear_fwd_epilogue(X, W, bias=torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="residual"):
        jf.linear_fwd_epilogue(X, W, residual=torch.zeros(64, 64))
    with pytest.raises(ValueError, match="contiguous"):
        jf.linear_fwd_epilogue(X, W, residual=torch.zeros(32, 64).t())
    with pytest.raises(ValueError, match="dtype"):
        jf.linear_fwd_epilogue(X, W, residual=torch.zeros(64, 32, dtype=torch.float64))
    with pytest.raises(ValueError, match="scales"):
        jf.bias_grad(jf.QTensor(X.q, torch.zeros(1, 3)))
    with pytest.raises(ValueError, match="codes"):
        jf.bias_grad(jf.QTensor(X.q.float(), X.s))
    qkv = q(32, 128)
    spec = jf.QKVRope(1, 20, 2, 1, 32, torch.zeros(32, 16), torch.zeros(32, 16))
    with pytest.raises(ValueError, match="layout"):
        jf.qkv_rope(qkv, spec._replace(layout="other"))
    with pytest.raises(ValueError, match="positions"):
        jf.qkv_rope(qkv, spec._replace(positions=torch.zeros(20, dtype=torch.int32)))
    with pytest.raises(ValueError, match="positions"):
        jf.qkv_rope(qkv, spec._replace(positions=torch.zeros(19, dtype=torch.int64)))
    with pytest.raises(ValueError, match="belong together"):
        jf.qkv_rope(qkv, spec._replace(sin=None))
    with pytest.raises(ValueError, match="gamma_q"):
        jf.qkv_rope(qkv, spec._replace(gamma_q=torch.ones(16)))
    with pytest.raises(ValueError, match="dk"):
        jf.qkv_rope_bwd(qkv, spec, torch.zeros(1, 20, 2, 32), torch.zeros(1, 20, 2, 32), torch.zeros(1, 20, 1, 32))
    with pytest.raises(ValueError, match="last dimension"):
        jf.qkv_rope_bwd(qkv, spec, torch.zeros(1, 20, 32, 2).transpose(2, 3), torch.zeros(1, 20, 1, 32), torch.zeros(1, 20, 1, 32))
    with pytest.raises(ValueError, match="missing"):
        jf.jf_qkv_rope_fwd(qkv, spec, torch.zeros(1, 20, 2, 32), None, torch.zeros(1, 20, 1, 32))


@pytest.mark.parametrize("name", B.ACTS)
def test_reference_derivatives_against_differences(name):
    """The 64-bit derivatives the GPU tests compare with, against central differences of the activations:
    the error of a central difference is h^2 / 6 |f'''| (third derivatives here are below 3) plus rounding
    2^-53 |f| / h."""
    x = torch.linspace(-9.0, 9.0, 4001, dtype=torch.float64) + 1e-3
    h = 1e-4
    diff = (B.act(x + h, name) - B.act(x - h, name)) / (2 * h)
    assert (B.act_grad(x, name) - diff).abs().max() <= h * h / 6 * 3 + 2.0 ** -52 * 9.1 / h


def test_reference_norm_backward_against_differences():
    g = torch.Generator().manual_seed(0)
    x, gamma = torch.randn(3, 2, 32, generator=g, dtype=torch.float64), torch.randn(32, generator=g, dtype=torch.float64)
    du, delta = torch.randn(3, 2, 32, generator=g, dtype=torch.float64), torch.randn(3, 2, 32, generator=g, dtype=torch.float64)
    h = 1e-5
    diff = ((B.rms(x + h * delta, gamma, 1e-6) - B.rms(x - h * delta, gamma, 1e-6)) * du).sum() / (2 * h)
    dx, terms = B.rms_backward(x, gamma, 1e-6, du)
    assert abs((dx * delta).sum() - diff) <= 1e-7 * (dx.abs() * delta.abs()).sum()
    dg = torch.randn(32, generator=g, dtype=torch.float64)
    diff = ((B.rms(x, gamma + h * dg, 1e-6) - B.rms(x, gamma - h * dg, 1e-6)) * du).sum() / (2 * h)
    assert abs((terms.sum((0, 1)) * dg).sum() - diff) <= 1e-9 * (terms.abs().sum((0, 1)) * dg.abs()).sum()
