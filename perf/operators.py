"""Measured cases of the operators that complete a transformer block around the INT8 linear layer.

Three families, each with its backward pass, on the tensors the library already trades in (INT8 codes
with one fp32 scale per 32x32 block):

* ``linear_fwd``   Z = act(X W^T + bias) + R, and ``linear_dgrad`` Z = (dY W) * act'(P) + R: the linear
                   layer with bias, activation and residual in its epilogue, with an INT8 or a dense result;
* ``bias_grad``    the column sums of an INT8 gradient;
* ``qkv_fwd``      per-head RMS norm of queries and keys and their rotary positions, from the INT8 output
                   of the QKV projection to the dense q, k, v that attention reads, and ``qkv_bwd``, its
                   gradient back into INT8 blocks.

With ``own`` false ``run`` computes the plain form in fp32 torch operations; with ``own`` true it makes
the calls a user makes. INT8 results are returned as the values they stand for, in bf16.
"""
import math

import torch

own = False

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
_TABLE = 32768          # positions of the rotary table a program keeps


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # fc1 of a GPT2-medium MLP in training: bias and GELU on chip, INT8 out, the pre-activation kept for the backward
        dict(name="fc1 bias gelu 4096x1024x4096", op="linear_fwd", M=4096, K=1024, N=4096, act="gelu", res="none", out="i8", pre=True),
        # fc2 of the hidden-4096 MLP: bias, and the residual stream held in bf16 (the largest product)
        dict(name="fc2 bias residual 8192x16384x4096", op="linear_fwd", M=8192, K=16384, N=4096, act="none", res="dense", out="bf16", pre=False),
        # the single 256-wide linear: a call whose latency counts
        dict(name="linear bias silu 256x256x256", op="linear_fwd", M=256, K=256, N=256, act="silu", res="none", out="fp32", pre=False),
        # sizes that leave every tile ragged, INT8 residual
        dict(name="linear ragged 352x1056x544", op="linear_fwd", M=352, K=1056, N=544, act="gelu_tanh", res="i8", out="i8", pre=True),
        # the input gradient through fc2 and the GELU before it, GPT2-medium
        dict(name="fc2 dgrad gelu' 4096x1024x4096", op="linear_dgrad", M=4096, N=1024, K=4096, act="gelu", res="none", out="i8"),
        # the input gradient of the hidden-4096 fc1, joined with the residual branch's gradient
        dict(name="fc1 dgrad residual 8192x16384x4096", op="linear_dgrad", M=8192, N=16384, K=4096, act="none", res="dense", out="bf16"),
        # bias gradients: the hidden-4096 fc1, and a small layer
        dict(name="bias grad 8192x16384", op="bias_grad", M=8192, N=16384),
        dict(name="bias grad 512x1056", op="bias_grad", M=512, N=1056),
        # hidden 4096 in training: 4 sequences of 2048, grouped heads, norm and full rotation, [B, H, S, D] out
        dict(name="qkv norm rope 4x2048 32+8 heads d128", op="qkv_fwd", batch=4, seq=2048, hq=32, hkv=8, d=128, rot=128,
             layout="half", norm=True, packed=False, dtype="bf16", heads_first=True),
        # one new token for each of 5 sequences at far positions, half of the head rotated, interleaved pairs
        dict(name="qkv rope decode 5x1 32+8 heads d128", op="qkv_fwd", batch=5, seq=1, hq=32, hkv=8, d=128, rot=64,
             layout="interleaved", norm=False, packed=True, dtype="fp16", heads_first=False),
        # the backward of the hidden-4096 case, with both norm weights' gradients
        dict(name="qkv norm rope bwd 4x2048 32+8 heads d128", op="qkv_bwd", batch=4, seq=2048, hq=32, hkv=8, d=128, rot=128,
             layout="half", norm=True, packed=False, dtype="bf16", heads_first=True),
        # GPT2-medium heads, packed documents (positions restart), a token count that is no multiple of 32
        dict(name="qkv norm rope bwd 1x1001 16+4 heads d64", op="qkv_bwd", batch=1, seq=1001, hq=16, hkv=4, d=64, rot=64,
             layout="interleaved", norm=True, packed=True, dtype="bf16", heads_first=False),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_fwd", "linear_dgrad", "linear_dgrad", "bias_grad", "qkv_fwd", "qkv_fwd", "qkv_bwd", "qkv_bwd"])
    if op in ("linear_fwd", "linear_dgrad"):
        while True:
            M, N, K = (32 * _log_uniform(rng, 1, 400) for _ in range(3))
            if M * N * K <= 8192 * 16384 * 4096:
                break
        out = rng.choice(["i8", "i8", "bf16", "fp16", "fp32"])
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        res = rng.choice(["none", "i8" if out == "i8" else "dense"])
        c = dict(op=op, M=M, N=N, K=K, act=act, res=res, out=out)
        if op == "linear_fwd":
            c["pre"] = rng.random() < 0.5
        return c
    if op == "bias_grad":
        return dict(op=op, M=32 * _log_uniform(rng, 1, 1024), N=32 * _log_uniform(rng, 1, 512))
    d = rng.choice([32, 64, 96, 128, 160, 256])
    while True:
        batch, seq = _log_uniform(rng, 1, 64), _log_uniform(rng, 1, 8192)
        hq, hkv = _log_uniform(rng, 1, 64), _log_uniform(rng, 1, 16)
        if batch * seq * (hq + 2 * hkv) * d <= 8192 * 48 * 128:
            break
    return dict(op=op, batch=batch, seq=seq, hq=hq, hkv=hkv, d=d, rot=rng.choice([r for r in (16, 32, 64, d // 2, d) if r <= d]),
                layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.6, packed=rng.random() < 0.5,
                dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), heads_first=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------ inputs
def _blocks(x):
    r, c = x.shape
    return x.view(r // 32, 32, c // 32, 32)


def _quantize(x):
    """Codes and scales of a dense fp32 matrix: s = absmax / 127 per 32x32 block, round half to even."""
    b = _blocks(x)
    s = b.abs().amax(dim=(1, 3)) / 127.0
    safe = torch.where(s > 0, s, torch.ones_like(s))
    q = torch.clamp(torch.round(b / safe[:, None, :, None]), -127, 127).to(torch.int8)
    return q.reshape(x.shape), s


def _expand(s):
    return s.repeat_interleave(32, 0).repeat_interleave(32, 1)


def _normal(g, rows, cols, std=1.0, outliers=0, factor=1.0):
    x = torch.randn(rows, cols, generator=g, device="cuda") * std
    if outliers:
        x[:, torch.randperm(cols, generator=g, device="cuda")[:outliers]] *= factor
    return x


def _tokens(c):
    return c["batch"] * c["seq"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    op = case["op"]
    if op in ("linear_fwd", "linear_dgrad"):
        M, N, K = case["M"], case["N"], case["K"]
        rows, cols = (M, N) if op == "linear_fwd" else (M, K)
        st["w"] = _quantize(_normal(g, N, K, 0.02))
        if op == "linear_fwd":
            st["x"] = _quantize(_normal(g, M, K, 1.0, max(1, K // 100), 30.0))  # a few outlier channels
            st["bias"] = torch.randn(N, generator=g, device="cuda") * 0.1
        else:
            st["dy"] = _quantize(_normal(g, M, N, 1e-3))
            if case["act"] != "none":
                st["p"] = _quantize(_normal(g, M, K, 1.0))
        std = 1.0 if op == "linear_fwd" else 1e-3
        if case["res"] == "dense":
            st["r"] = _normal(g, rows, cols, std).to(_DT[case["out"]])
        elif case["res"] == "i8":
            st["r"] = _quantize(_normal(g, rows, cols, std))
    elif op == "bias_grad":
        st["dy"] = _quantize(_normal(g, case["M"], case["N"], 1e-3))
    else:
        T, d, rot = _tokens(case), case["d"], case["rot"]
        C = (case["hq"] + 2 * case["hkv"]) * d
        x = torch.zeros((T + 31) // 32 * 32, C, device="cuda")   # tokens fill whole blocks of 32 rows with zero rows
        x[:T] = torch.randn(T, C, generator=g, device="cuda")
        x[:T, ::61] *= 8.0                                       # channels that stand out
        st["x"] = _quantize(x)
        j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
        angle = torch.arange(_TABLE, device="cuda", dtype=torch.float64)[:, None] * (10000.0 ** (-2.0 * j / rot))
        st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
        if case["packed"]:      # documents packed after one another, or sequences that are at different places
            start = torch.randint(0, _TABLE - case["seq"] + 1, (case["batch"], 1), generator=g, device="cuda")
            st["pos"] = (start + torch.arange(case["seq"], device="cuda")).reshape(-1) % 20011
        if case["norm"]:
            st["gq"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
            st["gk"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        if op == "qkv_bwd":
            for n, h in (("dq", case["hq"]), ("dk", case["hkv"]), ("dv", case["hkv"])):
                st[n] = (torch.randn(_shape(case, h), generator=g, device="cuda") * 1e-2).to(_DT[case["dtype"]])
    return st


def _shape(c, heads):
    return (c["batch"], heads, c["seq"], c["d"]) if c["heads_first"] else (c["batch"], c["seq"], heads, c["d"])


# ------------------------------------------------------------------------------------------ plain form
def _act(x, act):
    if act == "relu":
        return torch.clamp(x, min=0.0)
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    return x


def _act_grad(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (x + 0.044715 * x * x * x))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * x * x)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-x))
        return sg * (1.0 + x * (1.0 - sg))
    return torch.ones_like(x)


def _value(t):
    return t[0].float() * _expand(t[1])


def _as_i8(z):
    """The values that the INT8 form of z stands for, in bf16."""
    return _value(_quantize(z)).to(torch.bfloat16)


def _rotated(x, cos, sin, rot, layout, back):
    """x [T, H, D] with its first `rot` dimensions rotated by the tokens' angles (`back`: by their negative)."""
    y = x.clone()
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    s = -sin if back else sin
    u, v = a * cos - b * s, b * cos + a * s
    if layout == "half":
        y[..., :rot // 2], y[..., rot // 2:rot] = u, v
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = u, v
    return y


def _angles(st):
    c = st["case"]
    at = st["pos"] if "pos" in st else torch.arange(c["seq"], device="cuda").repeat(c["batch"])
    return st["cos"][at][:, None, :], st["sin"][at][:, None, :]


def _heads(c, x):
    """[T, columns] to the q, k and v parts [T, heads, d]."""
    x = x[:_tokens(c)].view(_tokens(c), -1, c["d"])
    return x[:, :c["hq"]], x[:, c["hq"]:c["hq"] + c["hkv"]], x[:, c["hq"] + c["hkv"]:]


def _laid_out(c, x):
    x = x.view(c["batch"], c["seq"], x.shape[1], c["d"])
    return (x.transpose(1, 2) if c["heads_first"] else x).contiguous().to(_DT[c["dtype"]])


def _flat(c, x):
    return (x.transpose(1, 2) if c["heads_first"] else x).reshape(_tokens(c), -1, c["d"]).float()


def _qkv_fwd(st):
    c = st["case"]
    q, k, v = _heads(c, _value(st["x"]))
    cos, sin = _angles(st)
    out = []
    for x, gamma in ((q, st.get("gq")), (k, st.get("gk"))):
        if gamma is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma
        out.append(_laid_out(c, _rotated(x, cos, sin, c["rot"], c["layout"], False)))
    return out + [_laid_out(c, v)]


def _qkv_bwd(st):
    c = st["case"]
    q, k, _ = _heads(c, _value(st["x"]))
    cos, sin = _angles(st)
    parts, dgammas = [], []
    for x, dy, gamma in ((q, st["dq"], st.get("gq")), (k, st["dk"], st.get("gk"))):
        du = _rotated(_flat(c, dy), cos, sin, c["rot"], c["layout"], True)
        if gamma is not None:
            rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
            xhat = x * rstd
            dgammas.append((du * xhat).sum((0, 1)))
            gr = du * gamma
            du = rstd * (gr - xhat * (gr * xhat).mean(-1, keepdim=True))
        parts.append(du)
    full = torch.zeros(st["x"][0].shape, device="cuda")
    full[:_tokens(c)] = torch.cat(parts + [_flat(c, st["dv"])], 1).reshape(_tokens(c), -1)
    return [_as_i8(full)] + dgammas


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "bias_grad":
        return _value(st["dy"]).sum(0)
    if op == "qkv_fwd":
        return _qkv_fwd(st)
    if op == "qkv_bwd":
        return _qkv_bwd(st)
    out = []
    if op == "linear_fwd":
        p = _value(st["x"]) @ _value(st["w"]).t() + st["bias"]
        if c["pre"]:
            out.append(_as_i8(p))
        z = _act(p, c["act"])
    else:
        z = _value(st["dy"]) @ _value(st["w"])
        if "p" in st:
            z = z * _act_grad(_value(st["p"]), c["act"])
    if c["res"] != "none":
        z = z + (st["r"].float() if c["res"] == "dense" else _value(st["r"]))
    return [_as_i8(z) if c["out"] == "i8" else z.to(_DT[c["out"]])] + out


# ------------------------------------------------------------------------------------------ the library's calls
def _library(st):
    import int8_fully_quantized_b200 as jf
    c = st["case"]
    op = c["op"]
    if op == "bias_grad":
        return jf.bias_grad(jf.QTensor(*st["dy"]))
    if op in ("qkv_fwd", "qkv_bwd"):
        spec = jf.QKVRope(c["batch"], c["seq"], c["hq"], c["hkv"], c["d"], st["cos"], st["sin"], positions=st.get("pos"),
                          gamma_q=st.get("gq"), gamma_k=st.get("gk"), eps=1e-6, layout=c["layout"])
        x = jf.QTensor(*st["x"])
        if op == "qkv_fwd":
            return list(jf.qkv_rope(x, spec, dtype=_DT[c["dtype"]], heads_first=c["heads_first"]))
        dx, dgq, dgk = jf.qkv_rope_bwd(x, spec, st["dq"], st["dk"], st["dv"], heads_first=c["heads_first"])
        return [jf.dequantize_block(dx)] + ([dgq, dgk] if c["norm"] else [])
    r = st.get("r")
    kw = dict(act=c["act"], residual=jf.QTensor(*r) if c["res"] == "i8" else r, out_dtype=None if c["out"] == "i8" else _DT[c["out"]])
    if op == "linear_fwd":
        y = jf.linear_fwd_epilogue(jf.QTensor(*st["x"]), jf.QTensor(*st["w"]), bias=st["bias"], want_pre=c["pre"], **kw)
        ys = list(y) if c["pre"] else [y]
    else:
        ys = [jf.linear_dgrad_epilogue(jf.QTensor(*st["dy"]), jf.QTensor(*st["w"]), pre=jf.QTensor(*st["p"]) if "p" in st else None, **kw)]
    return [jf.dequantize_block(y) if isinstance(y, jf.QTensor) else y for y in ys]


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    i8 = 1 + 4 / 1024                                  # bytes of an INT8 element with its share of the scale
    size = {"i8": i8, "fp32": 4, "bf16": 2, "fp16": 2}
    if op == "bias_grad":
        return dict(bytes=case["M"] * case["N"] * i8 + 4 * case["N"], flops=2 * case["M"] * case["N"])
    if op in ("qkv_fwd", "qkv_bwd"):
        T, d, b = _tokens(case), case["d"], size[case["dtype"]]
        qk, v = T * (case["hq"] + case["hkv"]) * d, T * case["hkv"] * d
        angles = 8 * (T if case["packed"] else case["seq"]) * (case["rot"] // 2) + (8 * T if case["packed"] else 0)
        if op == "qkv_fwd":
            return dict(bytes=(qk + v) * (i8 + b) + angles + (8 * d if case["norm"] else 0), flops=(10 if case["norm"] else 5) * qk + v)
        return dict(bytes=(qk + v) * (i8 + b) + (qk * i8 + 16 * d if case["norm"] else 0) + angles, flops=(20 if case["norm"] else 6) * qk + 3 * v)
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear_fwd":
        z = M * N
        moved = (M * K + N * K) * i8 + 4 * N + (z * i8 if case["pre"] else 0)
    else:
        z = M * K
        moved = (M * N + N * K) * i8 + (z * i8 if case["act"] != "none" else 0)
    moved += z * size[case["out"]] * (1 if case["res"] == "none" else 2)
    return dict(bytes=moved, flops=2 * M * N * K)


# ------------------------------------------------------------------------------------------ 64 bits
def _wide(t):
    q, s = t
    r, c = q.shape
    return (q.double().view(r // 32, 32, c // 32, 32) * s.double()[:, None, :, None]).view(r, c)


def _coded(z):
    """The values q s of the 32x32 block quantization of z, in 64 bits."""
    r, c = z.shape
    b = z.view(r // 32, 32, c // 32, 32).transpose(1, 2)
    s = b.abs().flatten(2).max(-1).values[..., None, None] / 127
    q = torch.where(s > 0, b / s, torch.zeros_like(b)).round()
    return (q * s).transpose(1, 2).reshape(r, c)


def _f64(x, act):
    """act(x) and act'(x) in 64 bits."""
    if act == "relu":
        return x.relu(), (x > 0).double()
    if act == "gelu":
        phi = 0.5 * torch.erfc(-x / 2 ** 0.5)
        return x * phi, phi + x * torch.exp(-x * x / 2) / (2 * math.pi) ** 0.5
    if act == "gelu_tanh":       # 0.5 (1 + tanh u) = sigmoid(2 u)
        k = (2 / math.pi) ** 0.5
        sg = torch.sigmoid(2 * k * (x + 0.044715 * x ** 3))
        return x * sg, sg + x * sg * (1 - sg) * 2 * k * (1 + 3 * 0.044715 * x ** 2)
    if act == "silu":
        sg = torch.sigmoid(x)
        return x * sg, sg + x * sg * (1 - sg)
    return x, torch.ones_like(x)


def _turned(x, angle, rot, layout):
    """Rotation as a product of complex numbers; x [T, H, D], angle [T, 1, rot / 2] complex."""
    pairs = x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2) if layout == "half" else x[..., :rot].unflatten(-1, (rot // 2, 2))
    z = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * angle)
    z = z.transpose(-1, -2).flatten(-2) if layout == "half" else z.flatten(-2)
    return torch.cat([z, x[..., rot:]], -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "bias_grad":
        return torch.ones(case["M"], dtype=torch.float64, device="cuda") @ _wide(st["dy"])
    if op in ("linear_fwd", "linear_dgrad"):
        w, pre = _wide(st["w"]), []
        if op == "linear_fwd":
            p = torch.addmm(st["bias"].double(), _wide(st["x"]), w.t())
            pre = [_coded(p)] if case["pre"] else []
            z = _f64(p, case["act"])[0]
        else:
            z = _wide(st["dy"]).mm(w)
            if case["act"] != "none":
                z *= _f64(_wide(st["p"]), case["act"])[1]
        if case["res"] != "none":
            z += st["r"].double() if case["res"] == "dense" else _wide(st["r"])
        return [_coded(z) if case["out"] == "i8" else z] + pre
    B, S, d, T = case["batch"], case["seq"], case["d"], _tokens(case)
    x = _wide(st["x"])[:T].unflatten(1, (-1, d))
    cut = [case["hq"], case["hkv"], case["hkv"]]
    at = st["pos"] if case["packed"] else torch.arange(T, device="cuda") % S
    z = torch.complex(st["cos"].double()[at], st["sin"].double()[at])[:, None]
    gammas = [st["gq"].double(), st["gk"].double()] if case["norm"] else [None, None]
    if op == "qkv_fwd":
        out = []
        for part, gm in zip(x.split(cut, 1), gammas + [None]):
            if gm is not None:
                part = part * gm * (part.square().sum(-1, keepdim=True) / d + 1e-6).rsqrt()
            if len(out) < 2:
                part = _turned(part, z, case["rot"], case["layout"])
            part = part.unflatten(0, (B, S))
            out.append(part.movedim(2, 1) if case["heads_first"] else part)
        return out
    dx, dgs = [], []
    for n, part, gm in zip(("dq", "dk", "dv"), x.split(cut, 1), gammas + [None]):
        dy = st[n].double()
        dy = (dy.movedim(1, 2) if case["heads_first"] else dy).flatten(0, 1)
        if n != "dv":
            dy = _turned(dy, z.conj(), case["rot"], case["layout"])
        if gm is not None:
            norm = (part.square().sum(-1, keepdim=True) / d + 1e-6).sqrt()
            dgs.append(torch.einsum("thd,thd->d", dy, part / norm))
            # d/dx of x gamma / n, n^2 = mean(x^2) + eps
            dy = dy * gm / norm - part * (dy * gm * part).sum(-1, keepdim=True) / (d * norm ** 3)
        dx.append(dy)
    full = torch.cat([torch.cat(dx, 1).flatten(1), torch.zeros(st["x"][0].shape[0] - T, (case["hq"] + 2 * case["hkv"]) * d, dtype=torch.float64, device="cuda")])
    return [_coded(full)] + dgs
