"""A whole transformer block, forward and backward, through the library as a training program would run it:
LayerNorm, QKV projection with bias, qkv_rope, attention (16-bit in this method: here plain fp32 torch),
output projection joined with the residual stream, LayerNorm, fc1 with bias and GELU, fc2 joined with the
residual stream; then every gradient. Each stage is fed the previous GPU stage's output and compared with its
64-bit plain form on the same input, so the tolerances are the stages' own (see the tests of the operators)."""
import pytest
import torch

import int8_fully_quantized_b200 as jf

import block_ref as B
from gpu_common import GEMM_RTOL, assert_requant_close, check_status, host

pytestmark = pytest.mark.gpu

BATCH, SEQ, H, HQ, HKV, D, F = 2, 80, 256, 4, 2, 64, 1024
T = BATCH * SEQ


def _codes(t, z64, what):
    q, s = B.quantize(z64)
    assert_requant_close(host(t.q), host(t.s), q.cpu().numpy(), s.cpu().numpy(), what)


def _dense(y, z64, mag, what):
    tol = 1.13 * GEMM_RTOL * mag + 2.0 ** -18 * z64.abs() + B.HALF_STEP[y.dtype] * z64.abs() * 1.01 + 2.0 ** -18 * mag
    assert ((y.double() - z64).abs() <= tol).all(), what


def _attention(q, k, v):
    """[B, H, S, D] causal attention with shared key heads, in fp32 torch."""
    k, v = (t.repeat_interleave(HQ // HKV, 1) for t in (k, v))
    w = (q @ k.transpose(2, 3)) * D ** -0.5
    w = w.masked_fill(torch.ones(SEQ, SEQ, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
    return torch.softmax(w, -1) @ v


def test_transformer_block():
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
    val = lambda t: B.value(*t)
    W = {n: jf.quantize_block(rnd(*s, std=0.05)) for n, s in dict(qkv=((HQ + 2 * HKV) * D, H), o=(H, HQ * D), fc1=(F, H), fc2=(H, F)).items()}
    bias = {n: rnd(w.rows, std=0.1) for n, w in W.items()}
    ln = [(1 + rnd(H, std=0.1), rnd(H, std=0.1)) for _ in range(2)]
    gq, gk = 1 + rnd(D, std=0.1), 1 + rnd(D, std=0.1)
    spec = jf.QKVRope(BATCH, SEQ, HQ, HKV, D, *jf.rope_table(SEQ, jf.rope_frequencies(D)[0]), gamma_q=gq, gamma_k=gk)
    stream0 = rnd(T, H).to(torch.bfloat16)

    # ---- forward
    n1 = jf.layernorm_i8(jf.quantize_block(stream0), *ln[0])
    qkv = jf.linear_fwd_epilogue(n1, W["qkv"], bias["qkv"])
    _codes(qkv, val(n1) @ val(W["qkv"]).t() + bias["qkv"].double(), "qkv")
    q, k, v = jf.qkv_rope(qkv, spec, heads_first=True)
    qkv_in = [t.float().requires_grad_() for t in (q, k, v)]
    att = _attention(*qkv_in)
    att_q = jf.quantize_block(att.detach().transpose(1, 2).reshape(T, HQ * D).contiguous())
    stream1 = jf.linear_fwd_epilogue(att_q, W["o"], bias["o"], residual=stream0, out_dtype=torch.bfloat16)
    p = val(att_q) @ val(W["o"]).t() + bias["o"].double()
    _dense(stream1, p + stream0.double(), val(att_q).abs() @ val(W["o"]).abs().t() + stream0.double().abs(), "stream1")
    n2 = jf.layernorm_i8(jf.quantize_block(stream1), *ln[1])
    h, pre = jf.linear_fwd_epilogue(n2, W["fc1"], bias["fc1"], act="gelu", want_pre=True)
    p = val(n2) @ val(W["fc1"]).t() + bias["fc1"].double()
    _codes(pre, p, "fc1 pre")
    _codes(h, B.act(p, "gelu"), "fc1")
    stream2 = stream1.clone()
    jf.jf_linear_fwd_epilogue(h, W["fc2"], y=stream2, bias=bias["fc2"], residual=stream2)
    p = val(h) @ val(W["fc2"]).t() + bias["fc2"].double()
    _dense(stream2, p + stream1.double(), val(h).abs() @ val(W["fc2"]).abs().t() + stream1.double().abs(), "stream2")

    # ---- backward
    d2 = rnd(T, H, std=1e-2).to(torch.bfloat16)                        # gradient of the stream
    d2q = jf.quantize_block(d2)
    db2 = jf.bias_grad(d2q)
    dpre = jf.linear_dgrad_epilogue(d2q, W["fc2"], pre, "gelu")
    _codes(dpre, (val(d2q) @ val(W["fc2"])) * B.act_grad(val(pre), "gelu"), "fc1 pre gradient")
    db1, dw1 = jf.bias_grad(dpre), jf.linear_wgrad(dpre, n2)
    dn2 = jf.linear_dgrad_epilogue(dpre, W["fc1"])
    dln2, _, _ = jf.layernorm_i8_bwd(jf.quantize_block(stream1), dn2, ln[1][0])
    d1 = (d2.float() + jf.dequantize_block(dln2, torch.float32)).to(torch.bfloat16)
    d1q = jf.quantize_block(d1)
    datt = jf.linear_dgrad_epilogue(d1q, W["o"], out_dtype=torch.float32)
    _dense(datt, val(d1q) @ val(W["o"]), val(d1q).abs() @ val(W["o"]).abs(), "attention gradient")
    att.backward(datt.reshape(BATCH, SEQ, HQ, D).transpose(1, 2))
    dqkv, dgq, dgk = jf.qkv_rope_bwd(qkv, spec, *[t.grad.to(torch.bfloat16) for t in qkv_in], heads_first=True)
    x = val(qkv)[:T].reshape(T, -1, D)
    cos, sin = (t.double().repeat(BATCH, 1) for t in (spec.cos, spec.sin))
    parts, dgs = [], []
    for xs, t, gm in ((x[:, :HQ], qkv_in[0], gq), (x[:, HQ:HQ + HKV], qkv_in[1], gk)):
        du = B.rotate(t.grad.to(torch.bfloat16).transpose(1, 2).reshape(T, -1, D).double(), cos, sin, "half", back=True)
        dx, terms = B.rms_backward(xs, gm.double(), 1e-6, du)
        parts.append(dx)
        dgs.append(terms)
    parts.append(qkv_in[2].grad.to(torch.bfloat16).transpose(1, 2).reshape(T, -1, D).double())
    _codes(dqkv, torch.cat(parts, 1).reshape(T, -1), "qkv gradient")
    for got, terms in zip((dgq, dgk), dgs):
        assert ((got.double() - terms.sum((0, 1))).abs() <= GEMM_RTOL * terms.abs().sum((0, 1))).all()
    for got, t in ((db2, d2q), (db1, dpre), (jf.bias_grad(dqkv), dqkv)):
        assert ((got.double() - val(t).sum(0)).abs() <= 2.0 ** -18 * val(t).abs().sum(0)).all()
    dn1 = jf.linear_dgrad_epilogue(dqkv, W["qkv"], residual=None)
    dwq = jf.linear_wgrad(dqkv, n1)
    assert dn1.q.shape == (T, H) and dwq.q.shape == W["qkv"].q.shape and dw1.q.shape == W["fc1"].q.shape
    check_status()
