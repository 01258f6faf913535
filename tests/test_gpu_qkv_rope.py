"""GPU tests of the rotary tables, of qkv_rope and of its gradient against 64-bit plain forms.

Tolerances, fixed before the first run. With a norm, x r gamma takes the sum of D squares in fp32 (exact products
of codes, at most D / 8 + 5 roundings of positive terms, half of which reach the root), a division, a root and three
products: below 32 x 2^-24 relative for D <= 256; the rotation's two products and sum add three roundings of terms
no larger than |u_a c| + |u_b s|. So forward |y - y64| <= 36 x 2^-24 (|u_a c| + |u_b s|) plus half a step of
the output type. The gradient's codes follow the re-quantization rule of gpu_common (its error is below 1e-5 of a
block's absmax); the norm weights' gradients sum T H terms, each within 40 x 2^-24, in registers, shuffles and
fp64: within 1e-5 of the sum of magnitudes, as the GEMMs."""
import numpy as np
import pytest
import torch

import int8_fully_quantized_b200 as jf

import block_ref as B
from gpu_common import GEMM_RTOL, assert_requant_close, check_status, host

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _case(seed, batch, seq, hq, hkv, d, rot, layout, norm, packed, extra_rows=0, table=512):
    g = _gen(seed)
    T = batch * seq
    rows = (T + 31) // 32 * 32 + extra_rows
    x = torch.randn(rows, (hq + 2 * hkv) * d, generator=g, device="cuda")
    x[:, 3::53] *= 10.0
    qkv = jf.QTensor(*B.quantize(x))
    f, m = jf.rope_frequencies(rot, scaling="yarn", factor=4.0, original_length=128) if rot else ([], 1.0)
    cos, sin = jf.rope_table(table, f, m) if rot else (None, None)
    pos = torch.randint(0, table, (batch, seq), generator=g, device="cuda") if packed else None
    gq, gk = (1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)) if norm else (None, None)
    return qkv, jf.QKVRope(batch, seq, hq, hkv, d, cos, sin, pos, gq, gk, 1e-5, layout), g


def _parts(v, a):
    T = a.batch * a.seq
    x = v[:T].reshape(T, -1, a.head_dim)
    return x[:, :a.q_heads], x[:, a.q_heads:a.q_heads + a.kv_heads], x[:, a.q_heads + a.kv_heads:]


def _angles(a):
    T = a.batch * a.seq
    at = a.positions.reshape(-1) if a.positions is not None else torch.arange(T, device="cuda") % max(a.seq, 1)
    if a.cos is None:
        z = torch.zeros(T, 0, dtype=torch.float64, device="cuda")
        return z, z
    return a.cos.double()[at], a.sin.double()[at]


def _laid(x, a, first):
    x = x.reshape(a.batch, a.seq, -1, a.head_dim)
    return x.transpose(1, 2) if first else x


def _forward64(qkv, a):
    """[(y, scale of its rounding)] for q, k, v as [T, H, D]."""
    cos, sin = _angles(a)
    out = []
    for x, gm in zip(_parts(B.value(*qkv), a), (a.gamma_q, a.gamma_k, None)):
        if len(out) == 2:
            out.append((x, x.abs()))
            continue
        u = B.rms(x, gm.double(), a.eps) if gm is not None else x
        out.append((B.rotate(u, cos, sin, a.layout), B.rotate(u.abs(), cos.abs(), -sin.abs(), a.layout).abs() +
                    B.rotate(u.abs(), cos.abs(), sin.abs(), a.layout).abs()))
    return out


def _check_forward(outs, qkv, a, first):
    for name, y, (ref, mag) in zip("qkv", outs, _forward64(qkv, a)):
        ref, mag = _laid(ref, a, first), _laid(mag, a, first)
        tol = 36 * B.EPS32 * mag + B.HALF_STEP[y.dtype] * ref.abs() * (1 + 2.0 ** -7) + B.TINY[y.dtype]
        assert y.shape == ref.shape
        if y.numel():
            assert ((y.double() - ref).abs() - tol).max().item() <= 0, name


CASES = [  # batch, seq, hq, hkv, d, rot, layout, norm, packed
    (1, 1, 1, 1, 32, 32, "half", False, False),
    (1, 1, 4, 2, 128, 128, "half", True, True),
    (3, 1, 8, 2, 64, 32, "interleaved", False, True),
    (1, 33, 3, 1, 96, 96, "half", True, False),
    (2, 47, 2, 2, 96, 48, "interleaved", True, True),
    (2, 64, 5, 3, 32, 16, "interleaved", True, False),
    (1, 129, 2, 1, 160, 80, "half", True, True),
    (1, 70, 2, 1, 192, 192, "interleaved", True, False),
    (2, 31, 3, 2, 256, 128, "half", True, False),
    (1, 257, 12, 4, 64, 64, "half", True, True),
    (1, 40, 2, 2, 64, 0, "half", True, False),
    (1, 40, 0, 2, 64, 64, "half", True, False),
    (2, 20, 4, 0, 64, 64, "interleaved", False, False),
    (1, 500, 13, 4, 128, 64, "interleaved", True, False),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_forward(case, dtype):
    for first in (False, True):
        qkv, a, _ = _case(sum(case[:6]), *case)
        _check_forward(jf.qkv_rope(qkv, a, DT[dtype], first), qkv, a, first)
    check_status()


def _backward64(qkv, a, dq, dk, dv, first):
    cos, sin = _angles(a)
    T = a.batch * a.seq
    full = torch.zeros(qkv.q.shape, dtype=torch.float64, device="cuda")
    parts, dgs = [], []
    for x, dy, gm in zip(_parts(B.value(*qkv), a), (dq, dk, dv), (a.gamma_q, a.gamma_k, None)):
        dy = (dy.transpose(1, 2) if first else dy).reshape(T, -1, a.head_dim).double()
        if len(parts) < 2:
            dy = B.rotate(dy, cos, sin, a.layout, back=True)
        if gm is not None:
            dy, terms = B.rms_backward(x, gm.double(), a.eps, dy)
            dgs.append(terms)
        parts.append(dy)
    full[:T] = torch.cat(parts, 1).reshape(T, -1)
    return full, dgs


def _grads(a, g, dtype, first, std=1e-2):
    shape = lambda n: (a.batch, n, a.seq, a.head_dim) if first else (a.batch, a.seq, n, a.head_dim)
    return [(torch.randn(shape(n), generator=g, device="cuda") * std).to(dtype) for n in (a.q_heads, a.kv_heads, a.kv_heads)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_backward(case, dtype):
    first = dtype == "bf16"
    qkv, a, g = _case(1 + sum(case[:6]), *case, extra_rows=64)
    grads = _grads(a, g, DT[dtype], first)
    dx, dgq, dgk = jf.qkv_rope_bwd(qkv, a, *grads, heads_first=first)
    full, dgs = _backward64(qkv, a, *grads, first)
    q, s = B.quantize(full)
    assert_requant_close(host(dx.q), host(dx.s), q.cpu().numpy(), s.cpu().numpy(), "dqkv")
    assert not dx.q[a.batch * a.seq:].any()                              # padding rows are zero
    for dg, terms in zip((dgq, dgk), dgs):
        assert ((dg.double() - terms.sum((0, 1))).abs() <= GEMM_RTOL * terms.abs().sum((0, 1)) + 1e-30).all()
    again = jf.qkv_rope_bwd(qkv, a, *grads, heads_first=first)
    assert torch.equal(again[0].q, dx.q) and torch.equal(again[0].s, dx.s)     # deterministic
    if dgq is not None:
        assert torch.equal(again[1], dgq) and torch.equal(again[2], dgk)
    check_status()


def test_gradient_against_differences():
    """The directional derivative of sum(q dq + k dk + v dv) along random directions of x and of the norm
    weights, from the 64-bit forward's central differences (h = 1e-4: error h^2 / 6 of third derivatives of order
    one, relative 1e-7), against the GPU's gradient: the INT8 rounding of dx is at most s / 2 per element."""
    qkv, a, g = _case(9, 1, 64, 3, 2, 64, 32, "interleaved", True, True)
    dq, dk, dv = _grads(a, g, torch.float32, False, std=1.0)
    dx, dgq, dgk = jf.qkv_rope_bwd(qkv, a, dq, dk, dv)
    x = B.value(*qkv)
    cos, sin = _angles(a)

    def loss(x, gq, gk):
        q, k, v = _parts(x, a)
        q, k = B.rotate(B.rms(q, gq, a.eps), cos, sin, a.layout), B.rotate(B.rms(k, gk, a.eps), cos, sin, a.layout)
        return sum((y * t.reshape(y.shape).double()).sum() for y, t in ((q, dq), (k, dk), (v, dv)))

    gq, gk, h = a.gamma_q.double(), a.gamma_k.double(), 1e-4
    for seed in range(4):
        d = torch.randn(x.shape, generator=_gen(seed), device="cuda", dtype=torch.float64)
        diff = (loss(x + h * d, gq, gk) - loss(x - h * d, gq, gk)) / (2 * h)
        got = (B.value(*dx) * d).sum()
        step = dx.s.double().repeat_interleave(32, 0).repeat_interleave(32, 1) * 0.5
        assert (got - diff).abs() <= (d.abs() * step).sum() * (1 + 1e-3) + 1e-6 * (B.value(*dx) * d).abs().sum()
        e = torch.randn(64, generator=_gen(seed + 10), device="cuda", dtype=torch.float64)
        for which, dg in ((0, dgq), (1, dgk)):
            up, dn = (loss(x, gq + t * e * (which == 0), gk + t * e * (which == 1)) for t in (h, -h))
            assert ((dg.double() * e).sum() - (up - dn) / (2 * h)).abs() <= 2e-5 * (dg.double().abs() * e.abs()).sum()


def test_strided_and_broadcast_tensors():
    """Outputs as slices of one packed [B, S, heads, D] buffer with guard heads; gradients as slices, expanded
    and transposed views."""
    qkv, a, g = _case(11, 2, 37, 4, 2, 64, 64, "half", True, False)
    ref = jf.qkv_rope(qkv, a, torch.bfloat16)
    buf = torch.full((2, 37, 10, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    jf.jf_qkv_rope_fwd(qkv, a, buf[:, :, 1:5], buf[:, :, 5:7], buf[:, :, 7:9])
    for got, want in zip((buf[:, :, 1:5], buf[:, :, 5:7], buf[:, :, 7:9]), ref):
        assert torch.equal(got, want)
    assert (buf[:, :, 0] == 3).all() and (buf[:, :, 9] == 3).all()
    # sequence-first memory seen as [B, H, S, D]; rows behind the tokens keep their bytes
    t = torch.full((40, 2, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    jf.jf_qkv_rope_fwd(qkv, a, t[:37].permute(1, 2, 0, 3), torch.empty(2, 2, 37, 64, dtype=torch.bfloat16, device="cuda"),
                       torch.empty(2, 2, 37, 64, dtype=torch.bfloat16, device="cuda"), heads_first=True)
    assert torch.equal(t[:37].permute(1, 0, 2, 3), ref[0]) and (t[37:] == 5).all()
    dq = torch.randn(2, 37, 10, 64, generator=g, device="cuda").to(torch.bfloat16)
    dv = torch.randn(1, 1, 1, 64, generator=g, device="cuda").to(torch.bfloat16).expand(2, 37, 2, 64)
    want = jf.qkv_rope_bwd(qkv, a, dq[:, :, :4].contiguous(), dq[:, :, 4:6].contiguous(), dv.contiguous())
    got = jf.qkv_rope_bwd(qkv, a, dq[:, :, :4], dq[:, :, 4:6], dv)
    assert torch.equal(got[0].q, want[0].q) and torch.equal(got[0].s, want[0].s) and torch.equal(got[1], want[1])
    check_status()


def test_positions_outside_the_table():
    """A bad position: NaN in the token's rotated dimensions, a zero gradient there, the other tokens
    untouched, and the status says so once."""
    qkv, a, g = _case(12, 1, 40, 2, 1, 64, 32, "half", False, True)
    good = jf.qkv_rope(qkv, a, torch.float32)
    grads = _grads(a, g, torch.float32, False)
    for bad in (-1, 512, 1 << 40):
        pos = a.positions.clone().reshape(-1)
        pos[17] = bad
        b = a._replace(positions=pos)
        q, k, v = jf.qkv_rope(qkv, b, torch.float32)
        assert jf.jf_device_status() == -11 and jf.jf_device_status() == 0
        for y, w in ((q, good[0]), (k, good[1])):
            assert torch.isnan(y[0, 17, :, :32]).all() and torch.equal(y[0, 17, :, 32:], w[0, 17, :, 32:])
            keep = [t for t in range(40) if t != 17]
            assert torch.equal(y[0, keep], w[0, keep])
        assert torch.equal(v, good[2])
        dx, _, _ = jf.qkv_rope_bwd(qkv, b, *grads)
        assert jf.jf_device_status() == -11 and jf.jf_device_status() == 0
        assert not dx.q[17, :32].any() and not dx.q[17, 64:96].any() and not dx.q[17, 128:160].any()
    with pytest.raises(jf.JetfireError):
        jf.qkv_rope(qkv, a._replace(positions=None, cos=a.cos[:39], sin=a.sin[:39]))


def test_zero_heads_tokens_and_zero_rows():
    qkv, a, _ = _case(13, 1, 32, 2, 1, 64, 64, "half", True, False)
    qkv.q[5] = 0                                                       # an all-zero token: the norm gives 0
    q, k, v = jf.qkv_rope(qkv, a, torch.float32)
    assert not q[0, 5].any() and not k[0, 5].any() and torch.isfinite(q).all()
    zero = jf.QTensor(torch.zeros_like(qkv.q), torch.zeros_like(qkv.s))
    dx, dgq, dgk = jf.qkv_rope_bwd(zero, a, *[torch.zeros_like(t) for t in (q, k, v)])
    assert not dx.q.any() and not dx.s.any() and not dgq.any() and not dgk.any()
    # no tokens: nothing written forward, a zero gradient backward
    none = a._replace(batch=0)
    assert jf.qkv_rope(qkv, none)[0].numel() == 0
    dx, dgq, dgk = jf.qkv_rope_bwd(qkv, none, *[torch.empty(0, 32, n, 64, device="cuda") for n in (2, 1, 1)])
    assert not dx.q.any() and not dx.s.any() and not dgq.any() and not dgk.any()
    check_status()


def test_streams_graphs_and_workspaces():
    qkv, a, g = _case(14, 2, 100, 8, 2, 64, 64, "half", True, False)
    grads = _grads(a, g, torch.bfloat16, False)
    ref, refb = jf.qkv_rope(qkv, a), jf.qkv_rope_bwd(qkv, a, *grads)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out, back = jf.qkv_rope(qkv, a), jf.qkv_rope_bwd(qkv, a, *grads)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, ref))
    assert torch.equal(back[0].q, refb[0].q) and torch.equal(back[1], refb[1]) and torch.equal(back[2], refb[2])
    # two captured backwards with workspaces of their own, replayed at the same time
    n = jf.jf_qkv_rope_bwd_workspace_bytes(qkv.rows, a)
    graphs = []
    for _ in range(2):
        dx, dgq, dgk = jf.empty_qtensor(qkv.rows, qkv.cols), torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            jf.jf_qkv_rope_bwd(qkv, a, *grads, dx, dgq, dgk, ws)
        graphs.append((graph, dx, dgq, dgk, torch.cuda.Stream()))
    for _ in range(5):
        for graph, dx, dgq, dgk, st in graphs:
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for graph, dx, dgq, dgk, st in graphs:
        assert torch.equal(dx.q, refb[0].q) and torch.equal(dgq, refb[1]) and torch.equal(dgk, refb[2])
    # only one of the weight gradients, and none
    dx, dgk = jf.empty_qtensor(qkv.rows, qkv.cols), torch.empty(64, device="cuda")
    jf.jf_qkv_rope_bwd(qkv, a, *grads, dx, None, dgk, torch.empty(n, dtype=torch.uint8, device="cuda"))
    assert torch.equal(dgk, refb[2]) and torch.equal(dx.q, refb[0].q)
    dx = jf.empty_qtensor(qkv.rows, qkv.cols)
    jf.jf_qkv_rope_bwd(qkv, a, *grads, dx)
    assert torch.equal(dx.q, refb[0].q) and torch.equal(dx.s, refb[0].s)
    check_status()


def test_offsets_past_32_bits():
    """Outputs more than 2^31 elements apart, and codes behind 2^31 bytes."""
    qkv, a, _ = _case(15, 2, 32, 2, 1, 128, 128, "half", True, False)
    ref = jf.qkv_rope(qkv, a)
    buf = torch.empty((1 << 31) + 64 * 1024, dtype=torch.bfloat16, device="cuda")
    q = torch.as_strided(buf, (2, 32, 2, 128), ((1 << 31) + 64, 256, 128, 1))
    jf.jf_qkv_rope_fwd(qkv, a, q, torch.empty_like(ref[1]), torch.empty_like(ref[2]))
    assert torch.equal(q, ref[0])
    del buf, q
    T, hq, d = 131104, 126, 128                                          # (126 + 2) * 128 * 131104 = 2^31 + 2^19
    one = torch.randint(-127, 128, (T, d), dtype=torch.int8, device="cuda", generator=_gen(3))
    big = jf.QTensor(one.repeat(1, hq + 2), torch.full((T // 32, (hq + 2) * d // 32), 0.01, device="cuda"))
    f, _ = jf.rope_frequencies(d)
    cos, sin = jf.rope_table(T, f)
    spec = jf.QKVRope(1, T, hq, 1, d, cos, sin)
    q, k, v = jf.qkv_rope(big, spec)
    small = jf.QTensor(one[-64:].repeat(1, 3).contiguous(), torch.full((2, 12), 0.01, device="cuda"))
    sq, sk, sv = jf.qkv_rope(small, jf.QKVRope(1, 64, 1, 1, d, cos, sin, torch.arange(T - 64, T, device="cuda")))
    assert torch.equal(q[:, -64:, :1], sq) and torch.equal(q[:, -64:, -1:], sq) and torch.equal(k[:, -64:], sk) and torch.equal(v[:, -64:], sv)
    check_status()


@pytest.mark.parametrize("length,half", [(1, 1), (7, 8), (4096, 64), (131072, 16)])
def test_rope_table(length, half):
    """cos and sin of fp64 angles, rounded once to fp32 (fp64's own error is far below half a step; the
    angle's rounding, up to 2^-53 of 131072 rad, adds 2^-36)."""
    f, m = jf.rope_frequencies(2 * half, scaling="linear", factor=1.0)
    cos, sin = jf.rope_table(length, f, 1.25)
    ang = torch.arange(length, dtype=torch.float64)[:, None] * torch.tensor(f, dtype=torch.float64)
    for got, ref in ((cos, 1.25 * ang.cos()), (sin, 1.25 * ang.sin())):
        assert ((got.cpu().double() - ref).abs() <= 2.0 ** -24 * ref.abs() * 1.001 + 2.0 ** -35).all()


def test_helpers_allocate_on_the_stream_they_run_on(monkeypatch):
    """The workspace that qkv_rope_bwd frees on return must not go to the next allocation of another stream while
    the kernels may still use it; the outputs of every helper equal those of the current stream."""
    g = torch.Generator(device="cuda").manual_seed(11)
    cos, sin = jf.rope_table(64, jf.rope_frequencies(64)[0])
    gamma = torch.ones(64, device="cuda")
    a = jf.QKVRope(2, 64, 4, 2, 64, cos, sin, gamma_q=gamma, gamma_k=gamma)
    x = jf.quantize_block(torch.randn(128, 512, device="cuda", generator=g))
    want = jf.qkv_rope(x, a)
    want_b = jf.qkv_rope_bwd(x, a, *want)
    side, seen, inner = torch.cuda.Stream(), [], jf._qkv_rope_bwd

    def spy(*args):
        seen.append((args[10].data_ptr(), args[10].numel(), torch.cuda.current_stream().cuda_stream))
        return inner(*args)

    monkeypatch.setattr(jf, "_qkv_rope_bwd", spy)
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        q, k, v = jf.qkv_rope(x, a, stream=s)
        dx, dgq, dgk = jf.qkv_rope_bwd(x, a, q, k, v, stream=s)
        ptr, n, on = seen[-1]
        later = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
        assert on == side.cuda_stream and all(t.data_ptr() != ptr for t in later)
        side.synchronize()
        for got, ref in zip((q, k, v, dx.q, dx.s, dgq, dgk), (*want, *want_b[0], *want_b[1:])):
            assert torch.equal(got, ref)
    c2, s2 = jf.rope_table(64, jf.rope_frequencies(64)[0], stream=side)
    side.synchronize()
    assert torch.equal(c2, cos) and torch.equal(s2, sin)
    check_status()
