"""The gated projections and the projection with an epilogue on the GPU, against 64-bit
references: every weight format, activation and optional part, odd and ragged sizes, one
token, last waves cut along K and along N, and the gradients."""
import pytest
import torch

from block_cases import ACT_ERR, BF, F32, LIPSCHITZ, Layer, act64, assert_within, frozen
from rank_linear_lora_b200 import autograd as LA
from rank_linear_lora_b200 import block
from rank_linear_lora_b200 import lora_linear as L

pytestmark = pytest.mark.gpu


def _bf(*shape):
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")


def _f32(*shape):
    return torch.full(shape, float("nan"), dtype=torch.float32, device="cuda")


# M, d_in, d_ff, r, format, activation
GLU = [
    (1, 8, 8, 8, "bf16", "silu"),            # the smallest of everything
    (1, 264, 136, 16, "bf16", "silu"),
    (3, 1000, 520, 24, "bf16", "gelu"),
    (16, 512, 264, 32, "bf16", "gelu_tanh"),
    (17, 512, 264, 32, "bf16", "relu"),
    (129, 200, 72, 72, "bf16", "silu"),      # a K tail of two 64-wide blocks
    (300, 328, 392, 16, "bf16", "none"),
    (257, 264, 1288, 8, "bf16", "gelu"),
    (1, 512, 136, 16, "q4", "silu"),
    (5, 448, 264, 16, "nf4", "silu"),
    (2, 272, 136, 8, "fp8", "gelu_tanh"),
    (300, 320, 264, 16, "q4", "silu"),
    (300, 336, 264, 16, "fp8", "gelu"),
    (300, 320, 392, 16, "nf4", "relu"),
    (1280, 2056, 2048, 16, "bf16", "silu"),  # 80 tiles, 33 K blocks: the last wave cut along K
    (1280, 264, 2048, 16, "bf16", "silu"),   # 5 K blocks: cut along N
    (1280, 2112, 2048, 16, "q4", "silu"),    # several tiles per CTA pair on a coded weight
    # fewer tiles than CTA pairs: every tile cut along K, in two or three pieces
    (33, 1040, 520, 16, "bf16", "silu"),
    (200, 4104, 264, 72, "bf16", "gelu"),
    (40, 4160, 264, 16, "q4", "silu"),
    (257, 4160, 136, 16, "nf4", "relu"),
    (129, 4112, 136, 72, "fp8", "silu"),
    (140, 1088, 72, 16, "q4", "none"),
]


def _glu_reference(y, act):
    h, err = y.h()
    f = y.n // 2
    g, u, eg, eu = h[:, :f], h[:, f:], err[:, :f], err[:, f:]
    a, _ = act64(g, act)
    ea = LIPSCHITZ * eg + ACT_ERR * g.abs()
    p = a * u
    ep = ea * (u.abs() + eu) + a.abs() * eu
    return h, err, p, ep + (BF + 2 * F32) * (p.abs() + ep)


@pytest.mark.parametrize("case", GLU, ids=["-".join(map(str, c)) for c in GLU])
@pytest.mark.parametrize("save", [False, True], ids=["plain", "saved"])
def test_glu_forward(case, save):
    M, d, f, r, fmt, act = case
    y = Layer(M, d, 2 * f, r, fmt, seed=11 + M)
    ws = L.act_workspace(y.wt.ops()[0], M, d, 2 * f, r)
    p, gu, xa = _bf(M, f), _bf(M, 2 * f) if save else None, _bf(M, r) if save else None
    n0 = L.lora_linear_launch_count()
    L.lora_glu_fwd(y.x, y.wt, y.A, y.B, p, gu, xa, y.alpha, act, ws)
    L.lora_linear_check(ws)
    assert L.lora_linear_launch_count() - n0 == 2
    h, err, want, bound = _glu_reference(y, act)
    assert_within("p", p, want, bound)
    if save:
        assert_within("gu", gu, h, err + BF * (h.abs() + err))
    again = _bf(M, f)
    L.lora_glu_fwd(y.x, y.wt, y.A, y.B, again, None, None, y.alpha, act, ws)
    L.lora_linear_check(ws)
    assert torch.equal(p, again)  # the same bits, and the workspace left ready for the next call


@pytest.mark.parametrize("M,d,f,r,fmt", [(200, 4104, 264, 72, "bf16"), (256, 4096, 512, 16, "bf16"), (130, 4096, 520, 16, "fp8")])
def test_k_cut_tiles_give_the_same_bits_every_time(M, d, f, r, fmt):
    """Few tiles and a long sum: each tile's pieces come from several CTA pairs, and warps of one
    tile add and read them side by side."""
    y = Layer(M, d, 2 * f, r, fmt, seed=5)
    ws = L.act_workspace(y.wt.ops()[0], M, d, 2 * f, r)
    n = 2 * f
    res, o = _bf(M, n), [_bf(M, n) for _ in range(2)]
    res.normal_()
    p = [_bf(M, f) for _ in range(2)]
    for i in range(100):
        L.lora_glu_fwd(y.x, y.wt, y.A, y.B, p[i > 0], None, None, y.alpha, "gelu", ws)
        L.lora_linear_act_fwd(y.x, y.wt, y.A, y.B, None, res, o[i > 0], None, None, y.alpha, "gelu", ws)
        assert torch.equal(p[0], p[i > 0]) and torch.equal(o[0], o[i > 0]), i
    L.lora_linear_check(ws)
    h, err, want, bound = _glu_reference(y, "gelu")
    assert_within("p", p[1], want, bound)


GLU_BWD = [
    (1, 264, 136, 16, "bf16", "silu"),
    (129, 200, 72, 72, "bf16", "gelu"),
    (300, 328, 392, 16, "bf16", "gelu_tanh"),
    (64, 136, 2056, 32, "bf16", "relu"),
    (200, 320, 264, 16, "q4", "silu"),
    (200, 336, 264, 16, "fp8", "silu"),
    (200, 320, 264, 16, "nf4", "none"),
]


@pytest.mark.parametrize("case", GLU_BWD, ids=["-".join(map(str, c)) for c in GLU_BWD])
def test_glu_backward_from_saved_values(case):
    """dGU and the layer's gradients from given pre-activations, xa saved or recomputed."""
    M, d, f, r, fmt, act = case
    y = Layer(M, d, 2 * f, r, fmt, seed=5 + M)
    gu, dP = y.randn(M, 2 * f), y.randn(M, f)
    gu[0, :8] = torch.tensor([0.0, -0.0, 30.0, -30.0, 64.0, -64.0, 1e-30, -1e-3], dtype=torch.bfloat16)
    xa = (y.s * (y.x.double() @ y.A.double().t())).to(torch.bfloat16)
    ws = L.workspace(y.wt.ops()[1], M, d, 2 * f, r)
    a, da = act64(gu[:, :f].double(), act)
    dh = torch.cat((dP.double() * gu[:, f:].double() * da, dP.double() * a), dim=1)
    scale = torch.cat((dP.double() * gu[:, f:].double(), dP.double() * gu[:, :f].double()), dim=1).abs()
    edh = BF * dh.abs() + 2 * ACT_ERR * LIPSCHITZ * (scale + dh.abs())
    ref = y.backward(dh, edh)
    for xa_save in (xa, None):
        dGU, dX, dA, dB = _bf(M, 2 * f), _bf(M, d), _f32(r, d), _f32(2 * f, r)
        L.lora_glu_bwd(dP, gu, y.x, y.wt, y.A, y.B, xa_save, dGU, dX, dA, dB, y.alpha, act, ws)
        L.lora_linear_check(ws)
        assert_within("dGU", dGU, dh, edh)
        for name, got, k in (("dX", dX, 3), ("dA", dA, 3), ("dB", dB, 3)):
            assert_within(name, got, *ref[name], roundings=k)


# M, d_in, d_out, r, format, activation, bias, residual
ACT = [
    (1, 8, 8, 8, "bf16", "none", False, False),
    (1, 264, 136, 16, "bf16", "none", False, True),
    (7, 1000, 520, 24, "bf16", "gelu", True, True),
    (16, 512, 264, 32, "bf16", "silu", True, False),
    (17, 512, 264, 32, "bf16", "gelu_tanh", False, True),
    (129, 200, 72, 72, "bf16", "relu", True, True),
    (300, 328, 392, 16, "bf16", "none", True, False),
    (1, 512, 136, 16, "q4", "none", True, True),
    (5, 448, 264, 16, "nf4", "silu", False, True),
    (2, 272, 136, 8, "fp8", "none", True, False),
    (300, 320, 264, 16, "q4", "gelu", True, True),
    (300, 336, 264, 16, "fp8", "none", False, True),
    (300, 320, 392, 16, "nf4", "relu", True, False),
    (1280, 2056, 4096, 16, "bf16", "gelu", True, True),  # 80 tiles: cut along K
    (1280, 264, 4104, 16, "bf16", "none", True, True),   # 85 tiles: cut along N
    (1280, 2112, 4096, 16, "fp8", "silu", True, True),
    (33, 1040, 520, 16, "bf16", "silu", True, True),      # cut along K in two or three pieces
    (200, 4104, 264, 72, "bf16", "none", False, True),
    (40, 4160, 264, 16, "q4", "gelu", True, True),
    (257, 4160, 136, 16, "nf4", "none", True, False),
    (129, 4112, 136, 72, "fp8", "silu", False, True),
]


def _act_reference(y, act, bias, residual):
    h, err = y.h()
    if bias:
        h, err = h + y.bias.double(), err + F32 * (h.abs() + y.bias.double().abs())
    a, _ = act64(h, act)
    ea = LIPSCHITZ * err + (0 if act == "none" else ACT_ERR * h.abs())
    out = a + y.residual.double() if residual else a
    return h, err, out, ea + (BF + 2 * F32) * (out.abs() + ea)


@pytest.mark.parametrize("case", ACT, ids=["-".join(map(str, c)) for c in ACT])
@pytest.mark.parametrize("save", [False, True], ids=["plain", "saved"])
def test_linear_act_forward(case, save):
    M, d, n, r, fmt, act, bias, residual = case
    y = Layer(M, d, n, r, fmt, seed=21 + M)
    ws = L.act_workspace(y.wt.ops()[0], M, d, n, r)
    out, pre, xa = _bf(M, n), _bf(M, n) if save else None, _bf(M, r) if save else None
    b, res = y.bias if bias else None, y.residual if residual else None
    L.lora_linear_act_fwd(y.x, y.wt, y.A, y.B, b, res, out, pre, xa, y.alpha, act, ws)
    L.lora_linear_check(ws)
    h, err, want, bound = _act_reference(y, act, bias, residual)
    assert_within("out", out, want, bound)
    if save:
        assert_within("pre", pre, h, err + BF * (h.abs() + err))
    again = _bf(M, n)
    L.lora_linear_act_fwd(y.x, y.wt, y.A, y.B, b, res, again, None, None, y.alpha, act, ws)
    L.lora_linear_check(ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("M,d,n,fmt", [(1, 264, 136, "bf16"), (16, 5064, 4112, "bf16"), (17, 520, 264, "bf16"),
                                       (33, 4104, 520, "bf16"), (300, 336, 392, "fp8"), (200, 4160, 264, "q4"),
                                       (1280, 2056, 4096, "bf16"), (1280, 264, 4104, "bf16")])
def test_residual_in_place(M, d, n, fmt):
    """out over residual: each element is read before it is written, by the thread that writes it."""
    y = Layer(M, d, n, 16, fmt, seed=61)
    ws = L.act_workspace(y.wt.ops()[0], M, d, n, 16)
    want = _bf(M, n)
    L.lora_linear_act_fwd(y.x, y.wt, y.A, y.B, y.bias, y.residual, want, None, None, y.alpha, "silu", ws)
    for _ in range(5):
        got = y.residual.clone()
        L.lora_linear_act_fwd(y.x, y.wt, y.A, y.B, y.bias, got, got, None, None, y.alpha, "silu", ws)
        assert torch.equal(got, want)
    L.lora_linear_check(ws)


ACT_BWD = [
    (1, 264, 136, 16, "bf16", "none", True),
    (1, 264, 8, 16, "bf16", "gelu", True),
    (33, 200, 1032, 72, "bf16", "gelu", True),
    (129, 200, 72, 16, "bf16", "silu", False),
    (700, 136, 264, 16, "bf16", "none", False),
    (1500, 136, 328, 8, "bf16", "relu", True),
    (200, 320, 264, 16, "q4", "gelu_tanh", True),
    (200, 336, 264, 16, "fp8", "silu", True),
    (200, 320, 264, 16, "nf4", "none", True),
]


@pytest.mark.parametrize("case", ACT_BWD, ids=["-".join(map(str, c)) for c in ACT_BWD])
def test_linear_act_backward_from_saved_values(case):
    M, d, n, r, fmt, act, bias = case
    y = Layer(M, d, n, r, fmt, seed=31 + M)
    pre, dOut = y.randn(M, n), y.randn(M, n)
    xa = (y.s * (y.x.double() @ y.A.double().t())).to(torch.bfloat16)
    ws = L.act_workspace(y.wt.ops()[1], M, d, n, r)
    _, da = act64(pre.double(), act)
    dh = dOut.double() * da
    e32 = torch.zeros_like(dh) if act == "none" else 2 * ACT_ERR * LIPSCHITZ * (dOut.double() * pre.double()).abs() + \
        2 * ACT_ERR * dOut.double().abs()
    edh = e32 if act == "none" else e32 + BF * (dh.abs() + e32)
    ref = y.backward(dh, edh)
    bits = None
    for _ in range(2):
        dPre, dX, dA, dB = _bf(M, n), _bf(M, d), _f32(r, d), _f32(n, r)
        db = _f32(n) if bias else None
        has = act != "none"
        L.lora_linear_act_bwd(dOut, pre if has else None, y.x, y.wt, y.A, y.B, xa, dPre if has else None, dX, dA, dB,
                              db, y.alpha, act, ws)
        L.lora_linear_check(ws)
        if has:
            assert_within("dPre", dPre, dh, edh)
        for name, got, k in (("dX", dX, 3), ("dA", dA, 3), ("dB", dB, 3)):
            assert_within(name, got, *ref[name], roundings=k)
        if bias:
            assert_within("dbias", db, dh.sum(0), e32.sum(0) + M * F32 * (dh.abs() + e32).sum(0))
            assert bits is None or torch.equal(db, bits)  # a fixed order of summation
            bits = db


def _autograd_reference(y, kind, act, bias, residual, dout):
    """Outputs and gradients by autograd in 64 bits."""
    leaf = {k: getattr(y, k).double().requires_grad_(True) for k in ("x", "A", "B")}
    if bias:
        leaf["bias"] = y.bias.double().requires_grad_(True)
    if residual:
        leaf["residual"] = y.residual.double().requires_grad_(True)
    h = leaf["x"] @ y.W.t() + y.s * (leaf["x"] @ leaf["A"].t()) @ leaf["B"].t()
    f = block._TORCH_ACT[act]
    if kind == "glu":
        out = f(h[:, :y.n // 2]) * h[:, y.n // 2:]
    else:
        h = h + leaf["bias"] if bias else h
        out = f(h) + leaf["residual"] if residual else f(h)
    return out.detach(), dict(zip(leaf, torch.autograd.grad(out, list(leaf.values()), dout.double())))


@pytest.mark.parametrize("fmt", ["bf16", "q4", "fp8", "nf4"])
@pytest.mark.parametrize("kind", ["glu", "act"])
def test_autograd_matches_the_formula(kind, fmt):
    """Through the autograd functions: leading dimensions, an input that is a strided view,
    gradients of every leaf.  Norm bounds: at most six independent roundings to bf16 lie
    between the inputs and a gradient (h or pre, dh, s.xa, s.g, the result, and the coded
    weight's own)."""
    M, d, n, r = 2 * 150, 320, 528, 16
    y = Layer(M, d, n, r, fmt, seed=3)
    x = torch.stack((y.x, y.x), dim=1)[:, 0].reshape(2, 150, d)  # rows 2 d apart
    x = x.detach().requires_grad_(True)
    A, B = y.A.clone().requires_grad_(True), y.B.clone().requires_grad_(True)
    f0, n0 = LA.fallback_calls, L.lora_linear_launch_count()
    if kind == "glu":
        out = block.lora_glu(x, y.wt, A, B, y.alpha, act="silu")
        dout = y.randn(2, 150, n // 2)
        leaves, names = (x, A, B), ("x", "A", "B")
    else:
        bias = y.bias.clone().requires_grad_(True)
        res = y.residual.reshape(2, 150, n).clone().requires_grad_(True)
        out = block.lora_linear_act(x, y.wt, A, B, y.alpha, bias=bias, residual=res, act="gelu")
        dout = y.randn(2, 150, n)
        leaves, names = (x, A, B, bias, res), ("x", "A", "B", "bias", "residual")
    grads = torch.autograd.grad(out, leaves, dout)
    torch.cuda.synchronize()
    assert LA.fallback_calls == f0 and L.lora_linear_launch_count() - n0 == 6
    want, gref = _autograd_reference(y, kind, "silu" if kind == "glu" else "gelu", kind == "act", kind == "act",
                                     dout.reshape(M, -1))
    lim = BF * (6 / 3) ** 0.5
    rel = lambda a, b: ((a.double().reshape(b.shape) - b).norm() / b.norm()).item()  # noqa: E731
    assert rel(out, want) <= lim
    for name, got in zip(names, grads):
        assert got.dtype == torch.bfloat16
        assert rel(got, gref[name]) <= lim, name


def test_no_grad_and_empty_batches():
    y = Layer(40, 64, 128, 8, seed=9)
    with torch.no_grad():
        a = block.lora_glu(y.x.requires_grad_(True), y.wt, y.A, y.B, y.alpha)
    b = block.lora_glu(y.x, y.wt, y.A, y.B, y.alpha)
    assert not a.requires_grad and b.requires_grad and torch.equal(a, b)
    x0 = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    A = y.A.clone().requires_grad_(True)
    for out in (block.lora_glu(x0, y.wt, A, y.B, y.alpha), block.lora_linear_act(x0, y.wt, A, y.B, y.alpha)):
        assert out.shape[0] == 0
        gx, gA = torch.autograd.grad(out.float().sum(), (x0, A))
        assert gx.shape == (0, 64) and not gA.any()


def test_infinities_and_nan_stay_in_their_rows():
    """A token with infinite or NaN inputs does not reach the other tokens' outputs."""
    y = Layer(140, 128, 144, 8, seed=17)
    ws = L.act_workspace(L.OP_FWD, 140, 128, 144, 8)
    clean, got = _bf(140, 144), _bf(140, 144)
    L.lora_linear_act_fwd(y.x, y.wt, y.A, y.B, y.bias, y.residual, clean, None, None, y.alpha, "gelu", ws)
    x = y.x.clone()
    x[3], x[70] = float("nan"), float("inf")
    L.lora_linear_act_fwd(x, y.wt, y.A, y.B, y.bias, y.residual, got, None, None, y.alpha, "gelu", ws)
    L.lora_linear_check(ws)
    rest = [i for i in range(140) if i not in (3, 70)]
    assert torch.equal(got[rest], clean[rest])
    assert got[3].isnan().all() and not got[70].isfinite().all()


def test_two_streams_and_two_graphs():
    """Calls on two streams, and two captured training steps replayed at the same time on
    new inputs, give what the calls give alone."""
    y = [Layer(300, 328, 1040, 16, seed=s) for s in (41, 42)]
    dout = [t.randn(300, 520) for t in y]

    def step(i, x):
        x = x.detach().requires_grad_(True)
        A, B = y[i].A.clone().requires_grad_(True), y[i].B.clone().requires_grad_(True)
        p = block.lora_glu(x, y[i].wt, A, B, y[i].alpha)
        return (p.detach(), *torch.autograd.grad(p, (x, A, B), dout[i]))

    alone = [step(i, y[i].x) for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got.append(step(i, y[i].x))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    graphs, xs, outs = [], [], []
    for i in (0, 1):
        xs.append(torch.zeros_like(y[i].x))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            outs.append(step(i, xs[i]))
        graphs.append(g)
    for i in (0, 1):
        xs[i].copy_(y[i].x)
    torch.cuda.synchronize()
    for _ in range(3):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


class Block(torch.nn.Module):
    """A transformer block on the framework's operators; attention itself, and the norms of x,
    in torch's own."""

    def __init__(self, d, hq, hk, D, f, r, g, fmts):
        super().__init__()
        self.ws = [frozen(fmt, n, k, g) for fmt, n, k in zip(fmts, ((hq + 2 * hk) * D, d, 2 * f, d), (d, hq * D, d, f))]
        W = [w[0] for w in self.ws]
        self.hq, self.hk, self.D, self.f = hq, hk, D, f
        self.qkv = block.LoraQKV(W[0], hq, hk, D, r, 2.0 * r, max_positions=128, rot=D // 2, theta=500.0)
        self.o = block._layer(W[1], r, 2.0 * r)
        self.mlp = block.LoraGatedMLP(W[2], W[3], r, 2.0 * r)
        with torch.no_grad():
            for B in (*(s.B_p(p) for s in (self.qkv, self.mlp.gate_up) for p in range(len(s.d_outs))), self.o.lora_B,
                      self.mlp.down.lora_B):
                B.copy_(torch.randn(B.shape, generator=g) * 0.3 / r ** 0.5)
            for w in (self.qkv.q_norm, self.qkv.k_norm):
                w.copy_(1 + 0.1 * torch.randn(D, generator=g))

    def attend(self, q, k, v, cast):
        k, v = (t.repeat_interleave(self.hq // self.hk, dim=2) for t in (k, v))
        s = torch.einsum("bihd,bjhd->bhij", cast(q), cast(k)) * self.D ** -0.5
        T = s.shape[-1]
        s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=s.device).triu(1), float("-inf"))
        return torch.einsum("bhij,bjhd->bihd", s.softmax(-1), cast(v)).flatten(2)

    def forward(self, x, pos):
        y = self.attend(*self.qkv(x, pos), torch.Tensor.float).to(torch.bfloat16)
        x = block.lora_linear_act(y, self.o._frozen(), self.o.lora_A, self.o.lora_B, self.o.alpha, residual=x)
        return self.mlp(x, residual=x)

    def trained(self):
        return {n: t for n, t in self.named_parameters() if t.requires_grad}

    def reference(self, x, pos):
        """(the leaves in 64 bits, the output)."""
        leaf = {n: t.detach().double().requires_grad_(True) for n, t in self.trained().items()}
        x64 = x.detach().double().requires_grad_(True)

        def lin(t, i, name):
            A, B = leaf[name + ".lora_A"], leaf[name + ".lora_B"]
            stack = {0: self.qkv, 2: self.mlp.gate_up}.get(i)
            if stack is not None:
                own = torch.zeros_like(B)
                for p, (a, b) in enumerate(stack.rows):
                    own[a:b, p * stack.r:(p + 1) * stack.r] = 1
                B = B * own
            return t @ self.ws[i][1].t() + 2.0 * (t @ A.t()) @ B.t()

        h = lin(x64, 0, "qkv.layer")
        c, s = (t.double()[pos][:, :, None] for t in (self.qkv.cos, self.qkv.sin))

        def heads(t, w):
            t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
            n = c.shape[-1]
            a, b = t[..., :n], t[..., n:2 * n]
            return torch.cat((a * c - b * s, b * c + a * s, t[..., 2 * n:]), -1)

        q, k, v = (t.unflatten(-1, (-1, self.D)) for t in h.split([e - b for b, e in self.qkv.rows], -1))
        y = self.attend(heads(q, leaf["qkv.q_norm"]), heads(k, leaf["qkv.k_norm"]), v, torch.Tensor.double)
        x1 = x64 + lin(y, 1, "o")
        gate, up = lin(x1, 2, "mlp.gate_up.layer").chunk(2, -1)
        return {"x": x64, **leaf}, x1 + lin(torch.nn.functional.silu(gate) * up, 3, "mlp.down")


@pytest.mark.parametrize("fmts", [("bf16",) * 4, ("nf4", "bf16", "q4", "fp8")], ids=["bf16", "coded"])
@pytest.mark.parametrize("T", [1, 37, 128])
def test_a_block_of_them_together(T, fmts):
    """Projections, norms with rotation, projection with residual, gated MLP: outputs and the
    gradients of x and every parameter, against autograd in 64 bits.  Some forty roundings to
    bf16 lie between x and a gradient (two of each operator's operands and one of its result,
    there and back), each of 2^-8 / sqrt(3) of a tensor's norm at most and independent:
    sqrt(40 / 3) 2^-8 = 1.4e-2 together, which the block (whose factors are of order one)
    may double."""
    g = torch.Generator().manual_seed(T)
    m = Block(256, 4, 2, 64, 320, 8, g, fmts)
    x = torch.randn(2, T, 256, generator=g).to(torch.bfloat16).cuda().requires_grad_(True)
    dout = torch.randn(2, T, 256, generator=g).to(torch.bfloat16).cuda()
    pos = torch.stack((torch.arange(T), torch.randint(0, 128, (T,), generator=g))).cuda()
    out = m(x, pos)
    names, leaves = zip(("x", x), *m.trained().items())
    grads = torch.autograd.grad(out, leaves, dout)
    leaf, want = m.reference(x, pos)
    gref = torch.autograd.grad(want, [leaf[n] for n in names], dout.double())
    def rel(a, b):
        return ((a.double() - b).norm() / b.norm()).item()
    assert rel(out, want.detach()) <= 3e-2
    for n, a, b in zip(names, grads, gref):
        if T == 1 and ("q_norm" in n or "k_norm" in n):
            assert a.float().abs().max() <= 1e-2  # one key: a softmax over one score has no gradient
        else:
            assert rel(a, b) <= 3e-2, n
    with torch.no_grad():  # the forward without autograd: nothing saved, the same bits
        assert torch.equal(m(x, pos), out)


def test_a_captured_step_of_the_block():
    """Forward, backward and a plain SGD step in one graph: replays give what eager steps give."""
    def model():
        torch.manual_seed(1)  # lora_A is drawn from the default generator
        return Block(256, 4, 2, 64, 320, 8, torch.Generator().manual_seed(3), ("bf16", "q4", "fp8", "bf16"))

    g = torch.Generator().manual_seed(5)
    xs = [torch.randn(1, 24, 256, generator=g).to(torch.bfloat16).cuda() for _ in range(3)]
    pos = torch.arange(24, device="cuda")[None]

    def step(m, x):
        out = m(x, pos)
        leaves = list(m.trained().values())
        grads = torch.autograd.grad(out.float().square().mean(), leaves)
        with torch.no_grad():
            for t, d in zip(leaves, grads):
                t.sub_(d, alpha=2.0 ** -6)
        return out.detach()

    eager = model()
    want = [step(eager, x) for x in xs]
    m, x = model(), torch.zeros_like(xs[0])
    keep = [t.detach().clone() for t in m.trained().values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(m, x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(m, x)
    with torch.no_grad():
        for t, k in zip(m.trained().values(), keep):
            t.copy_(k)
    for xi, w in zip(xs, want):
        x.copy_(xi)
        graph.replay()
        assert torch.equal(out, w)
    for a, b in zip(m.trained().values(), eager.trained().values()):
        assert torch.equal(a, b)


def test_which_gradients_are_asked_for():
    """Any subset of the inputs may want a gradient; the others get none, and the wanted ones are
    the same bits as when all are."""
    y = Layer(40, 64, 96, 8, seed=21)
    cos, sin = block.rope_table(64, 16, device="cuda")
    pos = torch.arange(40, device="cuda")
    wq, wk = (1 + 0.1 * y.randn(2, 32)).unbind(0)
    cases = [
        (lambda x, A, B, b, r: block.lora_linear_act(x, y.wt, A, B, y.alpha, bias=b, residual=r, act="silu"),
         [y.x, y.A, y.B, y.bias, y.residual], y.randn(40, 96)),
        (lambda x, A, B, r: block.lora_linear_act(x, y.wt, A, B, y.alpha, residual=r), [y.x, y.A, y.B, y.residual],
         y.randn(40, 96)),
        (lambda x, A, B: block.lora_glu(x, y.wt, A, B, y.alpha), [y.x, y.A, y.B], y.randn(40, 48)),
        (lambda q, k, a, b: torch.cat(block.qk_norm_rope(q, k, a, b, cos, sin, pos), 1),
         [y.randn(40, 3, 32), y.randn(40, 2, 32), wq, wk], y.randn(40, 5, 32)),
        (lambda q, k, b: torch.cat(block.qk_norm_rope(q, k, None, b), 1), [y.randn(40, 3, 32), y.randn(40, 2, 32), wk],
         y.randn(40, 5, 32)),
    ]
    for f, ins, up in cases:
        leaves = [t.clone().requires_grad_(True) for t in ins]
        whole = torch.autograd.grad(f(*leaves), leaves, up)
        for wanted in range(1, 1 << len(ins)):
            some = [t.clone().requires_grad_(bool(wanted >> i & 1)) for i, t in enumerate(ins)]
            f(*some).backward(up)
            for i, t in enumerate(some):
                assert (t.grad is None) if not wanted >> i & 1 else torch.equal(t.grad, whole[i]), (wanted, i)


def test_errors_of_the_native_side():
    """Types, shapes and devices by name; differentiating twice and inputs changed before the
    backward are errors; a call after them works."""
    y = Layer(24, 64, 96, 8, seed=22)
    cos, sin = block.rope_table(64, 16, device="cuda")
    q, k, pos = y.randn(24, 3, 32), y.randn(24, 2, 32), torch.arange(24, device="cuda")
    for match, f in [
        ("x:", lambda: block.lora_glu(y.x.float(), y.wt, y.A, y.B, 16.0)),
        ("A:", lambda: block.lora_glu(y.x, y.wt, y.A[:, :56], y.B, 16.0)),
        ("B:", lambda: block.lora_glu(y.x, y.wt, y.A, y.B.t(), 16.0)),
        ("bias:", lambda: block.lora_linear_act(y.x, y.wt, y.A, y.B, 16.0, bias=y.bias[:88])),
        ("residual:", lambda: block.lora_linear_act(y.x, y.wt, y.A, y.B, 16.0, residual=y.residual.half())),
        ("A:", lambda: block.lora_linear_act(y.x, y.wt, y.A.cpu(), y.B, 16.0)),
        ("rows", lambda: block.lora_glu(y.x, y.wt.tensors[0][:95], y.A, y.B[:95], 16.0)),
        ("W", lambda: block.lora_glu(y.x, y.wt.tensors[0].half(), y.A, y.B, 16.0)),
        ("q, k", lambda: block.qk_norm_rope(q, k[:23], None, None)),
        ("k:", lambda: block.qk_norm_rope(q, k.half(), None, None)),
        ("q, k", lambda: block.qk_norm_rope(q.double(), k.double(), None, None)),
        ("q_weight:", lambda: block.qk_norm_rope(q, k, torch.ones(31, dtype=torch.bfloat16, device="cuda"), None)),
        ("go together", lambda: block.qk_norm_rope(q, k, None, None, cos, None, pos)),
        ("sin:", lambda: block.qk_norm_rope(q, k, None, None, cos, sin[:, :4], pos)),
        ("positions:", lambda: block.qk_norm_rope(q, k, None, None, cos, sin, pos[:23])),
        ("positions:", lambda: block.qk_norm_rope(q, k, None, None, cos, sin, pos.int())),
    ]:
        with pytest.raises(ValueError, match=match):
            f()
    with pytest.raises(L.LoraError, match="lora_qk_norm_rope_fwd") as e:
        block.qk_norm_rope(q, k, None, None, eps=-1.0)
    assert e.value.status == 1
    with pytest.raises(L.LoraError, match="lora_linear_act_fwd"):
        block.lora_linear_act(y.x, y.wt, y.A, y.B, float("inf"))
    x = y.x.clone().requires_grad_(True)
    for f in (lambda: block.lora_glu(x, y.wt, y.A, y.B, 16.0), lambda: block.lora_linear_act(x, y.wt, y.A, y.B, 16.0)):
        up = torch.ones_like(f()).requires_grad_(True)
        g, = torch.autograd.grad(f(), x, up, create_graph=True)
        with pytest.raises(RuntimeError, match="twice"):
            g.sum().backward()
        out = f()
        with torch.no_grad():
            x.add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.backward(up)
        f().backward(up.detach())
    assert x.grad is not None


def test_threads_and_many_shapes():
    """Calls from two threads on streams of their own, over more shapes than workspaces are kept,
    give what the calls give alone."""
    import threading
    y = Layer(90, 64, 96, 8, seed=23)
    alone = [block.lora_glu(y.x[:m], y.wt, y.A, y.B, y.alpha) for m in range(1, 91)]
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(3):
                for m in range(1, 91):
                    if not torch.equal(block.lora_glu(y.x[:m], y.wt, y.A, y.B, y.alpha), alone[m - 1]):
                        bad.append(m)

    ts = [threading.Thread(target=work) for _ in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_threads_on_one_stream():
    """Forwards and backwards from two threads on one stream (their backwards in the threads
    themselves, not one after the other in autograd's own) do not mix up each other's workspace."""
    import threading
    y = [Layer(70, 264, 400, 16, seed=s) for s in (24, 25)]
    up = y[0].randn(70, 400)

    def step(i):
        x, A, B = (t.clone().requires_grad_(True) for t in (y[i].x, y[i].A, y[i].B))
        out = block.lora_linear_act(x, y[i].wt, A, B, y[i].alpha, act="silu")
        return (out.detach(), *torch.autograd.grad(out, (x, A, B), up))

    alone = [step(i) for i in (0, 1)]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        with torch.autograd.set_multithreading_enabled(False):
            for _ in range(60):
                got[i].append(step(i))

    ts = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    for i in (0, 1):
        assert len(got[i]) == 60 and all(torch.equal(a, b) for g in got[i] for a, b in zip(g, alone[i]))


# A few tokens.  x does not fit into shared memory whole: several segments of it (the last one
# shorter), one group of rows per CTA or more than share a segment, the last batch not full.
# M, d_in, d_out, r, format
FEW = [
    (8, 13000, 1008, 16, "bf16"),
    (16, 5064, 9616, 24, "bf16"),
    (9, 20040, 144, 8, "bf16"),
    (3, 28672, 272, 16, "bf16"),
    (2, 65544, 80, 8, "bf16"),
    (16, 5056, 9616, 24, "q4"),
    (8, 12992, 5008, 16, "q4"),
    (5, 20032, 272, 16, "q4"),
    (16, 5056, 9616, 24, "nf4"),
    (7, 12992, 5008, 16, "nf4"),
    (16, 5072, 9616, 16, "fp8"),
    (6, 20016, 1008, 16, "fp8"),
    # groups of 32 rows, x whole and in segments, the last group with a first half only
    (12, 520, 4112, 16, "bf16"),
    (16, 5064, 4112, 24, "bf16"),
    (4, 512, 4112, 16, "q4"),
    (13, 576, 4112, 16, "q4"),
    (8, 12992, 4112, 16, "q4"),
    (7, 576, 4112, 16, "nf4"),
    (8, 13056, 4112, 16, "nf4"),
    (1, 528, 4112, 16, "fp8"),
    (11, 528, 4112, 16, "fp8"),
    (8, 13088, 4112, 16, "fp8"),
]


@pytest.mark.parametrize("case", FEW, ids=["-".join(map(str, c)) for c in FEW])
def test_few_tokens_of_many_values(case):
    M, d, n, r, fmt = case
    y = Layer(M, d, n, r, fmt, seed=50 + M)
    ws = L.act_workspace(y.wt.ops()[0], M, d, n, r)
    want = {"out": _act_reference(y, "silu", True, True)[2:], "p": _glu_reference(y, "silu")[2:]}
    first = None
    for _ in range(3):
        got = {"out": _bf(M, n), "p": _bf(M, n // 2)}
        L.lora_linear_act_fwd(y.x, y.wt, y.A, y.B, y.bias, y.residual, got["out"], None, None, y.alpha, "silu", ws)
        L.lora_glu_fwd(y.x, y.wt, y.A, y.B, got["p"], None, None, y.alpha, "silu", ws)
        L.lora_linear_check(ws)
        first = first or got
        for name, t in got.items():
            assert torch.equal(t, first[name])
    for name, t in first.items():
        assert_within(name, t, *want[name])
