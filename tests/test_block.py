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


def _h(data=0x1000, ts=1024, hs=128, heads=8):
    return ctypes.byref(L.lora_heads_t(data, ts, hs, heads))


def test_qk_norm_rope_refusals(lib):
    def fwd(dtype=0, q=_h(), k=None, wq=None, cos=0x2000, sin=0x3000, pos=0x4000, n_pos=16, qo=_h(0x5000), ko=None, M=4,
            D=128, rot=128, inter=0, eps=1e-6):
        return lib.lora_qk_norm_rope_fwd(dtype, q, k, P(wq), None, P(cos), P(sin), P(pos), n_pos, qo, ko, M, D, rot, inter,
                                         1, eps, None)

    bad = [dict(dtype=3), dict(dtype=-1), dict(q=None), dict(q=None, qo=None), dict(qo=None), dict(ko=_h()), dict(M=0),
           dict(M=(1 << 30) + 1), dict(D=0), dict(D=132), dict(D=264), dict(rot=132), dict(rot=136), dict(rot=-8),
           dict(rot=12), dict(eps=-1.0), dict(eps=float("nan")), dict(cos=None), dict(sin=None), dict(pos=None),
           dict(n_pos=0), dict(q=_h(None)), dict(q=_h(heads=0)), dict(q=_h(heads=5000)), dict(qo=_h(heads=7)),
           dict(q=_h(ts=120)), dict(q=_h(hs=120)), dict(q=_h(hs=-128)), dict(qo=_h(ts=512)), dict(qo=_h(ts=0))]
    for b in bad:
        assert fwd(**b) == 1, b
    for b in (dict(q=_h(0x1008)), dict(qo=_h(0x5002)), dict(q=_h(ts=1028)), dict(q=_h(hs=132, ts=2048)),
              dict(wq=0x6004), dict(cos=0x2008), dict(sin=0x3004), dict(pos=0x4004)):
        assert fwd(**b) == 2, b

    def bwd(dy=_h(0x7000), q=_h(), dq=_h(0x5000), dwq=None, dwk=None, ws=None, nws=0):
        return lib.lora_qk_norm_rope_bwd(0, dy, None, q, None, None, None, P(0x2000), P(0x3000), P(0x4000), 16, dq, None,
                                         P(dwq), P(dwk), 4, 128, 128, 0, 1, 1e-6, P(ws), nws, None)

    assert bwd(dy=None) == 1 and bwd(dq=None) == 1 and bwd(dwk=0x8000) == 1 and bwd(q=None) == 1
    assert bwd(dwq=0x8000) == 4 and bwd(dwq=0x8000, ws=0x10000, nws=256) == 4
    assert bwd(dwq=0x8000, ws=0x10010, nws=1 << 30) == 2 and bwd(dwq=0x8004, ws=0x10000, nws=1 << 30) == 2
    assert L.lora_qk_norm_rope_workspace_size(4, 8, 128) > 0
    for bad in ((0, 8, 128), (4, 0, 128), (4, 8, 12), (4, 8, 264)):
        assert L.lora_qk_norm_rope_workspace_size(*bad) == 0


def test_rope_table_far_positions():
    """Angles of far positions keep their digits: against Python's own 64-bit arithmetic."""
    import math
    cos, sin = block.rope_table(40000, 16, theta=500.0)
    assert cos.dtype == torch.float32 and cos.shape == (40000, 8)
    for p, i in ((0, 0), (1, 7), (39999, 0), (39999, 5), (31234, 2)):
        a = p * 500.0 ** (-2 * i / 16)
        assert abs(cos[p, i].item() - math.cos(a)) < 1e-6 and abs(sin[p, i].item() - math.sin(a)) < 1e-6


@pytest.mark.parametrize("interleaved", [False, True])
def test_unfused_heads(interleaved, monkeypatch):
    """LORA_LINEAR_FUSED=0: torch's composition of the norms and the rotation, on q, k and on
    the stacked projection, which gives the same q and k and v as it is."""
    monkeypatch.setenv("LORA_LINEAR_FUSED", "0")
    g = torch.Generator().manual_seed(2)
    h = torch.randn(2, 6, (3 + 2 * 2) * 16, generator=g).requires_grad_(True)
    wq, wk = torch.randn(16, generator=g), torch.randn(16, generator=g)
    cos, sin = block.rope_table(32, 8)
    pos = torch.randint(0, 32, (2, 6), generator=g)
    q, k, v = block.qkv_heads(h, 3, 2, 16, wq, wk, cos, sin, pos, interleaved=interleaved)
    q2, k2 = block.qk_norm_rope(h[..., :48].unflatten(-1, (3, 16)), h[..., 48:80].unflatten(-1, (2, 16)), wq, wk, cos,
                                sin, pos, interleaved=interleaved)
    assert torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(v, h[..., 80:].unflatten(-1, (2, 16)))
    n = h.detach()[1, 3, 16:32].double()
    n = n / (n.square().mean() + 1e-6).sqrt() * wq.double()
    i, j = (2, 3) if interleaved else (1, 5)
    c, s = cos[pos[1, 3], 1].double(), sin[pos[1, 3], 1].double()
    assert abs(q[1, 3, 1, i].item() - (n[i] * c - n[j] * s).item()) < 1e-5
    assert abs(q[1, 3, 1, j].item() - (n[j] * c + n[i] * s).item()) < 1e-5
    assert abs(q[1, 3, 1, 9].item() - n[9].item()) < 1e-5
    (q.sum() + k.sum() + v.sum()).backward()
    assert h.grad is not None
    with pytest.raises(ValueError, match="columns"):
        block.qkv_heads(h, 3, 3, 16)


def test_workspace_sizes(lib):
    """The backward's workspace holds the bias partials besides the layer's; the forward's, its own
    hand-over of tiles cut along K, if any."""
    for op in range(8):
        layer = L.lora_linear_workspace_size(op, 512, 1024, 768, 16)
        own = L.lora_linear_act_workspace_size(op, 512, 1024, 768, 16)
        assert own >= layer + 768 * 4 if op % 2 else own > 0
    # 16 tiles of 256 x 256 for 256 tokens of 4096 columns: three pieces of each, two of them handed over
    cut = L.lora_linear_act_workspace_size(L.OP_FWD, 256, 4096, 4096, 8)
    assert cut >= 2 * 16 * 256 * 256 * 4
    assert cut == L.lora_linear_act_workspace_size(L.OP_FWD_Q4, 256, 4096, 4096, 8)
    # a few tokens cut nothing
    assert L.lora_linear_act_workspace_size(L.OP_FWD, 16, 4096, 4096, 8) < 1 << 20
    assert L.lora_linear_act_workspace_size(8, 512, 1024, 768, 16) == 0
    assert L.lora_linear_act_workspace_size(0, 0, 1024, 768, 16) == 0
    assert L.lora_linear_act_workspace_size(1, 1, 8, 8, 8) > 0


def test_bindings_refuse_what_they_cannot_pass():
    x, W = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(32, 16, dtype=torch.bfloat16)
    A, Bm = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(32, 8, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):  # CPU tensors (RuntimeError where there is no CUDA device at all)
        L.lora_glu_fwd(x, W, A, Bm, torch.zeros(4, 16, dtype=torch.bfloat16), None, None, 16.0, "silu", None)
    with pytest.raises(ValueError, match="act"):
        block.lora_glu(x, W, A, Bm, 16.0, act="swish")
    with pytest.raises(ValueError, match="residual"):
        block.lora_linear_act(x, W, A, Bm, 16.0, residual=torch.zeros(3, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="W"):
        L._weight(torch.zeros(4, dtype=torch.bfloat16), 0)


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


def test_modules_unfused(monkeypatch):
    """The stacked projections and the modules over them on the unfused compositions: each
    projection with its own adapter, no gradient and no change outside their blocks."""
    monkeypatch.setenv("LORA_LINEAR_FUSED", "0")
    g = torch.Generator().manual_seed(4)

    def bf(*s):
        return (torch.randn(*s, generator=g) / s[-1] ** 0.5).to(torch.bfloat16)

    qkv = block.LoraQKV(bf(4 * 16 + 2 * 16, 32), hq=2, hk=2, D=16, r=8, alpha=16.0, max_positions=64, rot=8)
    mlp = block.LoraGatedMLP(bf(48, 32), bf(40, 24), r=8, alpha=16.0, act="gelu")
    for stack in (qkv, mlp.gate_up):
        for p in range(len(stack.d_outs)):
            with torch.no_grad():
                stack.B_p(p).copy_(bf(*stack.B_p(p).shape))
    x = (4 * bf(2, 3, 32)).requires_grad_(True)
    pos = torch.arange(3).expand(2, 3)
    h = block.LoraProjections.forward(qkv, x)
    W = qkv.layer.weight.double()
    for p, (a, b) in enumerate(qkv.rows):
        w = W[a:b] + 2.0 * qkv.B_p(p).detach().double() @ qkv.A_p(p).detach().double()
        torch.testing.assert_close(h[..., a:b].double(), x.detach().double() @ w.t(), rtol=4e-2, atol=4e-2)
    q, k, v = qkv(x, pos)
    assert q.shape == (2, 3, 2, 16) and torch.equal(v, h[..., 64:].unflatten(-1, (2, 16)))
    assert torch.equal(q[:, 0, :, 8:], block.qk_norm_rope(h[..., :32].unflatten(-1, (2, 16)), h[..., 32:64].unflatten(
        -1, (2, 16)), qkv.q_norm, qkv.k_norm)[0][:, 0, :, 8:])
    out = mlp(x, residual=torch.ones(2, 3, 40, dtype=torch.bfloat16))
    assert out.shape == (2, 3, 40)
    opt = torch.optim.SGD([t for m in (qkv, mlp) for t in m.parameters() if t.requires_grad], lr=0.1)
    (q.float().square().sum() + k.float().sum() + v.float().sum() + out.float().sum()).backward()
    opt.step()
    for stack in (qkv, mlp.gate_up):
        B, G = stack.layer.lora_B.detach().clone(), stack.layer.lora_B.grad.clone()
        assert G.any()
        for p, (a, b) in enumerate(stack.rows):
            for t in (B, G):
                t[a:b, p * 8:(p + 1) * 8] = 0
        assert not B.any() and not G.any()
    assert qkv.q_norm.grad is not None and mlp.down.lora_A.grad is not None and x.grad is not None
    qkv.to(torch.float64)
    assert qkv.cos.dtype == torch.float32
    with pytest.raises(ValueError, match="positions"):
        qkv(x)
    with pytest.raises(ValueError, match="rows"):
        block.LoraProjections(bf(48, 32), (24, 16), r=8)
    with pytest.raises(ValueError, match="down takes"):
        block.LoraGatedMLP(bf(48, 32), bf(40, 32))
    with pytest.raises(ValueError, match="exact"):
        block.LoraProjections(bf(48, 32), (16, 16, 16), r=8, alpha=16777217.0 / 16777216.0 * 3.0 + 1e-6)


def test_head_strides_beyond_any_memory(lib):
    """Offsets that would pass 63 bits are refused, not wrapped around."""
    far = 1 << 40

    def fwd(q, qo, M):
        return lib.lora_qk_norm_rope_fwd(0, q, None, None, None, P(0x2000), P(0x3000), P(0x4000), 16, qo, None, M, 128, 128, 0, 1,
                                         1e-6, None)

    for M in (1 << 30, (1 << 23) + 1, 1 << 24):
        for hs in (128, far):
            assert fwd(_h(ts=far, hs=hs), _h(0x5000), M) == 1
            assert fwd(_h(), _h(0x5000, ts=far, hs=hs), M) == 1
