"""Inputs, 64-bit references and error bounds for the operators around the layer.

The bounds are sums of the roundings that the operators take, each at most half a step of
its type relative to the value (bf16: 2^-8, fp16: 2^-11, fp32: 2^-24), carried through the
formulas with absolute values; an fp32 sum of K terms adds at most K * 2^-24 of the sum of
the terms' absolute values.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from rank_linear_lora_b200.autograd import FrozenWeight

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
BF, F32 = HALF[torch.bfloat16], HALF[torch.float32]
# the fp32 activations: a few units in the last place from __expf, __fdividef and erff, each
# relative to a value of at most 1.2 (|v| <= 64 in the tests: e^v's argument rounds by 2^-18)
ACT_ERR = 2.0 ** -17
LIPSCHITZ = 1.2  # |act'| <= 1.13 for each activation

CODEBOOK = np.array([-1.0, -0.7, -0.52, -0.39, -0.28, -0.18, -0.09, 0.0, 0.08, 0.16, 0.25, 0.34, 0.44, 0.56, 0.72, 1.0],
                    dtype=np.float32)


def frozen(fmt, n, d, g, device="cuda"):
    """(FrozenWeight, its exact fp64 value, the relative rounding its use takes)."""
    def rand(*s):
        return torch.rand(*s, generator=g).to(device)

    if fmt == "bf16":
        w = (torch.randn(n, d, generator=g) / d ** 0.5).to(torch.bfloat16).to(device)
        return FrozenWeight("bf16", (w,)), w.double(), 0.0
    if fmt == "fp8":
        q = (torch.randn(n, d, generator=g) * 64).clamp_(-448, 448).to(torch.float8_e4m3fn).to(device)
        sc = ((1 + rand(n)) / (64 * d ** 0.5)).to(torch.bfloat16)
        return FrozenWeight("fp8", (q.view(torch.uint8), sc)), q.double() * sc.double()[:, None], BF
    q = torch.randint(1, 16, (n, d), generator=g).to(device)
    sc = ((1 + rand(n, d // 64)) / d ** 0.5).to(torch.bfloat16)
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8).contiguous()
    wide = sc.double().repeat_interleave(64, dim=1)
    if fmt == "q4":
        return FrozenWeight("q4", (packed, sc)), (q.double() - 8) * wide / 7, BF
    cb = torch.from_numpy(CODEBOOK).double().to(device)
    return FrozenWeight("nf4", (packed, sc), codebook=CODEBOOK), cb[q] * wide, BF


def act64(v, act):
    """(act(v), act'(v)) in 64 bits."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        return v.clamp(min=0), (v > 0).double()
    if act == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * (1 - s)
    if act == "gelu":
        c = 0.5 * torch.erfc(-v / math.sqrt(2))
        return v * c, c + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)


class Layer:
    """Inputs of one (stacked) layer and its fp64 quantities."""

    def __init__(self, M, d, n, r, fmt="bf16", alpha=32.0, seed=0, b_std=0.3, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def bf(t):
            return t.to(torch.bfloat16).to(device)

        self.M, self.d, self.n, self.r, self.alpha, self.s = M, d, n, r, alpha, alpha / r
        self.g = g
        self.x = bf(torch.randn(M, d, generator=g))
        self.wt, self.W, self.w_err = frozen(fmt, n, d, g, device)
        self.A = bf(torch.randn(r, d, generator=g) / d ** 0.5)
        self.B = bf(torch.randn(n, r, generator=g) * b_std / r ** 0.5)
        self.bias = bf(torch.randn(n, generator=g))
        self.residual = bf(torch.randn(M, n, generator=g))

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g).to(torch.bfloat16).to(self.x.device)

    def h(self):
        """(h, bound of the fp32 accumulator's error)."""
        x, A, B = self.x.double(), self.A.double(), self.B.double()
        sxa = self.s * (x @ A.t())
        h = x @ self.W.t() + sxa @ B.t()
        mag = x.abs() @ self.W.abs().t()
        sxa_mag = abs(self.s) * (x.abs() @ A.abs().t())
        sxa_err = BF * sxa.abs() + 2 * self.d * F32 * sxa_mag
        err = self.w_err * mag + 2 * (self.d + self.r) * F32 * (mag + sxa_mag @ B.abs().t()) + sxa_err @ B.abs().t()
        return h, err

    def backward(self, dY, dY_err):
        """{name: (value, bound)} of the layer's gradients for the exact dY, when the layer
        is given a dY off by at most dY_err; dA, dB before any rounding to 16 bits."""
        x, A, B, s = self.x.double(), self.A.double(), self.B.double(), self.s
        sxa = s * (x @ A.t())
        sxa_err = BF * sxa.abs() + 2 * self.d * F32 * abs(s) * (x.abs() @ A.abs().t())
        sg = s * (dY @ B)
        ady = dY.abs() + dY_err
        sg_err = BF * sg.abs() + abs(s) * (dY_err @ B.abs()) + 2 * self.n * F32 * abs(s) * (ady @ B.abs())
        asg = sg.abs() + sg_err
        dX = dY @ self.W + sg @ A
        big = ady @ self.W.abs()
        dX_err = (dY_err @ self.W.abs() + self.w_err * big + sg_err @ A.abs()
                  + 2 * (self.n + self.r) * F32 * (big + asg @ A.abs()))
        dX_err = dX_err + BF * (dX.abs() + dX_err)
        dA = sg.t() @ x
        dA_err = sg_err.t() @ x.abs() + 2 * self.M * F32 * (asg.t() @ x.abs())
        dB = dY.t() @ sxa
        dB_err = dY_err.t() @ sxa.abs() + ady.t() @ sxa_err + 2 * self.M * F32 * (ady.t() @ sxa.abs())
        return {"dX": (dX, dX_err), "dA": (dA, dA_err), "dB": (dB, dB_err)}


def assert_within(name, got, want, bound, roundings=None):
    """Every element within its bound; and, for values made of many rounded terms, the norm
    of the error within that of `roundings` independent bf16 roundings (each uniform over a
    half step either way: half step / sqrt(3) of rms)."""
    got = got.detach().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    over = (got - want).abs() - bound
    worst = over.max().item() if over.numel() else 0.0
    assert not torch.isnan(over).any(), f"{name}: NaN"
    assert worst <= 0, f"{name}: {worst:.3e} over its bound at {tuple(np.unravel_index(int(over.argmax()), got.shape))}"
    if roundings and want.numel() > 4096:
        rel = ((got - want).norm() / want.norm()).item()
        assert rel <= BF * math.sqrt(roundings / 3), f"{name}: relative error {rel:.3e}"
