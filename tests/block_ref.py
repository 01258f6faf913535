"""Plain 64-bit forms of the transformer-block operators (linear epilogues, bias gradient, QKV norm and
rotation), written from their formulas with torch float64 on whatever device the inputs are, and the
quantized inputs the tests share. Nothing here uses the library."""
import math

import torch

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS32 = 2.0 ** -24          # half a unit in the last place of fp32, relative
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}   # half a subnormal step


def blocks(x):
    r, c = x.shape
    return x.reshape(r // 32, 32, c // 32, 32)


def quantize(x):
    """(codes, scales) of a dense matrix, s = absmax / 127 per 32x32 block in fp32, round half to even."""
    b = blocks(x.float())
    s = b.abs().amax((1, 3)) / torch.full((), 127.0, device=x.device)
    safe = torch.where(s > 0, s, torch.ones_like(s))
    q = torch.where(s[:, None, :, None] > 0, torch.round(b / safe[:, None, :, None]).clamp(-127, 127), torch.zeros_like(b))
    return q.to(torch.int8).reshape(x.shape), s


def value(q, s):
    return (blocks(q.double()) * s.double()[:, None, :, None]).reshape(q.shape)


def act(x, name):
    if name == "relu":
        return x.clamp(min=0)
    if name == "gelu":
        return x * 0.5 * torch.erfc(-x / math.sqrt(2.0))
    if name == "gelu_tanh":
        return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
    if name == "silu":
        return x * torch.sigmoid(x)
    return x


def act_grad(x, name):
    if name == "relu":
        return (x > 0).to(x.dtype)
    if name == "gelu":
        return 0.5 * torch.erfc(-x / math.sqrt(2.0)) + x * torch.exp(-x * x / 2) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        k = 2.0 * math.sqrt(2.0 / math.pi)
        g = torch.sigmoid(k * (x + 0.044715 * x ** 3))
        return g + x * g * (1 - g) * k * (1 + 3 * 0.044715 * x * x)
    if name == "silu":
        g = torch.sigmoid(x)
        return g + x * g * (1 - g)
    return torch.ones_like(x)


def rotate(x, cos, sin, layout, back=False):
    """x [T, H, D]; cos, sin [T, rot / 2] float64."""
    half = cos.shape[-1]
    c, s = cos[:, None], (-sin if back else sin)[:, None]
    y = x.clone()
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    return y


def rms(x, gamma, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma


def rms_backward(x, gamma, eps, du):
    """(dx, the terms of dgamma [T, H, D]) of u = rms(x)."""
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xhat, g = x * r, du * gamma
    return r * (g - xhat * (g * xhat).mean(-1, keepdim=True)), du * xhat
