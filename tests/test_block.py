"""The operators around the layer on the CPU: argument checks of the C entry points (all
before any device work), of the Python binding, workspace sizes, and the unfused
compositions they fall back to when asked."""
import ctypes

import pytest
import torch

from rank_linear_lora_b200 import autograd as LA
from rank_linear_lora_b200 import block
from rank_linear_lora_b200 import build as B
from rank_linear_lora_b200 import lora_linear as L

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load_library()


def _w(fmt=0, data=0x2000, scale=None, codebook=None):
    return L.lora_weight_t(fmt, data, scale, codebook)


def _glu(lib, w=None, x=0x1000, A=0x3000, B_=0x4000, p=0x5000, gu=None, xa=None, M=64, di=256, f=128, r=8, alpha=16.0,
         act=2, ws=0x10000, nws=1 << 30):
    w = _w() if w is None else w
    return lib.lora_glu_fwd(P(x), ctypes.byref(w) if w else None, P(A), P(B_), P(p), P(gu), P(xa), M, di, f, r, alpha,
                            act, P(ws), nws, None)


def test_glu_forward_refusals(lib):
    """INVALID_ARG 1, MISALIGNED 2: every case fails before any pointer is used."""
    bad = dict(x=None), dict(A=None), dict(B_=None), dict(p=None), dict(w=False), dict(w=_w(data=None)), \
        dict(w=_w(fmt=4)), dict(w=_w(fmt=-1)), dict(w=_w(fmt=1)), dict(w=_w(fmt=3, scale=0x2800)), dict(M=0), \
        dict(di=250), dict(f=0), dict(f=4), dict(f=132), dict(f=(1 << 23) + 8), dict(r=12), dict(r=264), \
        dict(alpha=float("inf")), dict(act=5), dict(act=-1), dict(w=_w(fmt=1, scale=0x2800), di=96), \
        dict(w=_w(fmt=2, scale=0x2800), di=264)
    for b in bad:
        assert _glu(lib, **b) == 1, b
    for b in dict(x=0x1008), dict(w=_w(data=0x2004)), dict(p=0x5002), dict(gu=0x6008), dict(xa=0x6004), \
            dict(w=_w(fmt=1, scale=0x2808)):
        assert _glu(lib, **b) == 2, b


def test_glu_backward_refusals(lib):
    def bwd(dP=0x1000, gu=0x1100, x=0x1200, A=0x3000, B_=0x4000, dGU=0x5000, dX=None, dA=0x6000, dB=0x7000, act=2, f=128):
        w = _w()
        return lib.lora_glu_bwd(P(dP), P(gu), P(x), ctypes.byref(w), P(A), P(B_), None, P(dGU), P(dX), P(dA), P(dB), 64,
                                256, f, 8, 16.0, act, P(0x10000), 1 << 30, None)

    for b in dict(dP=None), dict(gu=None), dict(dGU=None), dict(dGU=0x1100), dict(x=None), dict(A=None), dict(dA=None), \
            dict(dB=None), dict(act=9), dict(f=12):
        assert bwd(**b) == 1, b
    for b in dict(dP=0x1004), dict(gu=0x1108), dict(dGU=0x5008), dict(dX=0x8008), dict(dA=0x6004):
        assert bwd(**b) == 2, b


def test_linear_act_refusals(lib):
    def fwd(bias=None, res=None, out=0x5000, pre=None, act=0, di=256, do=128, w=None):
        w = _w() if w is None else w
        return lib.lora_linear_act_fwd(P(0x1000), ctypes.byref(w), P(0x3000), P(0x4000), P(bias), P(res), P(out), P(pre),
                                       None, 64, di, do, 8, 16.0, act, P(0x10000), 1 << 30, None)

    for b in dict(out=None), dict(act=5), dict(di=4), dict(do=20), dict(w=_w(fmt=7)):
        assert fwd(**b) == 1, b
    for b in dict(bias=0x8002), dict(res=0x8008), dict(pre=0x8004), dict(out=0x5004):
        assert fwd(**b) == 2, b

    def bwd(dOut=0x1000, pre=0x1100, dPre=0x1200, dbias=None, dA=0x6000, act=3, nws=1 << 30, ws=0x10000):
        w = _w()
        return lib.lora_linear_act_bwd(P(dOut), P(pre), P(0x1300), ctypes.byref(w), P(0x3000), P(0x4000), None, P(dPre),
                                       None, P(dA), P(0x7000), P(dbias), 64, 256, 128, 8, 16.0, act, P(ws), nws, None)

    for b in dict(dOut=None), dict(pre=None), dict(dPre=None), dict(dPre=0x1000), dict(dPre=0x1100), dict(dA=None), \
            dict(act=6):
        assert bwd(**b) == 1, b
    for b in dict(dOut=0x1008), dict(pre=0x1108), dict(dPre=0x1208), dict(dbias=0x9004):
        assert bwd(**b) == 2, b


def test_workspace_sizes(lib):
    """The forward's workspace is the layer's; the backward's holds the bias partials too."""
    for op in range(8):
        layer = L.lora_linear_workspace_size(op, 512, 1024, 768, 16)
        own = L.lora_linear_act_workspace_size(op, 512, 1024, 768, 16)
        assert own == layer if op % 2 == 0 else own >= layer + 768 * 4
    assert L.lora_linear_act_workspace_size(8, 512, 1024, 768, 16) == 0
    assert L.lora_linear_act_workspace_size(0, 0, 1024, 768, 16) == 0
    assert L.lora_linear_act_workspace_size(1, 1, 8, 8, 8) > 0


def test_bindings_refuse_what_they_cannot_pass():
    x, W = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(32, 16, dtype=torch.bfloat16)
    A, Bm = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(32, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # CPU tensors
        L.lora_glu_fwd(x, W, A, Bm, torch.zeros(4, 16, dtype=torch.bfloat16), None, None, 16.0, "silu", None)
    with pytest.raises(ValueError, match="act"):
        block.lora_glu(x, W, A, Bm, 16.0, act="swish")
    with pytest.raises(ValueError, match="residual"):
        block.lora_linear_act(x, W, A, Bm, 16.0, residual=torch.zeros(3, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="W"):
        L._weight(torch.zeros(4, dtype=torch.bfloat16))


@pytest.mark.parametrize("act", sorted(L.ACTIVATIONS))
def test_unfused_compositions(act, monkeypatch):
    """LORA_LINEAR_FUSED=0: torch's composition, with gradients of every leaf."""
    monkeypatch.setenv("LORA_LINEAR_FUSED", "0")
    g = torch.Generator().manual_seed(1)

    def bf(*s):
        return torch.randn(*s, generator=g).to(torch.bfloat16)

    x, W, A, Bm = bf(2, 5, 24), bf(48, 24) / 5, bf(8, 24) / 5, bf(48, 8) / 3
    bias, res = bf(48), bf(2, 5, 48)
    for t in (x, A, Bm, bias, res):
        t.requires_grad_(True)
    n0 = LA.fallback_calls
    p = block.lora_glu(x, W, A, Bm, 16.0, act=act)
    o = block.lora_linear_act(x, W, A, Bm, 16.0, bias=bias, residual=res, act=act)
    assert LA.fallback_calls == n0 + 2 and p.shape == (2, 5, 24) and o.shape == (2, 5, 48)
    xs = x.detach().double()
    h = xs @ W.double().t() + 2.0 * (xs @ A.detach().double().t()) @ Bm.detach().double().t()
    f = block._TORCH_ACT[act]
    torch.testing.assert_close(p.double(), f(h[..., :24]) * h[..., 24:], rtol=4e-2, atol=4e-2)
    torch.testing.assert_close(o.double(), f(h + bias.detach().double()) + res.detach().double(), rtol=4e-2, atol=6e-2)
    (p.float().sum() + o.float().sum()).backward()
    assert all(t.grad is not None for t in (x, A, Bm, bias, res)) and W.grad is None
