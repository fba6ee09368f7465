"""The operators around the layer at their edges: what a caller may pass and rarely does."""
import os
import subprocess
import sys

import pytest
import torch

from block_cases import F32, HALF, Layer, act64, assert_within
from rank_linear_lora_b200 import block
from rank_linear_lora_b200 import lora_linear as L

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bf(*shape):
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")


def _heads_inputs(M, hq, hk, D, rot, seed=0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(M, (hq + 2 * hk) * D, generator=g).to(dtype).cuda()
    w = (1 + 0.1 * torch.randn(2, D, generator=g)).to(dtype).cuda()
    cos, sin = block.rope_table(64, rot, device="cuda")
    return h, w[0], w[1], cos, sin, torch.randint(0, 64, (M,), generator=g).cuda()


def _split(h, hq, hk, D):
    return h[:, :hq * D].unflatten(1, (hq, D)), h[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))


@pytest.mark.parametrize("grad", [True, False], ids=["grad", "no_grad"])
def test_forward_mode_is_an_error(grad):
    """Tangents do not go through the kernels: a dual tensor is refused (not computed without its
    tangent), with gradients enabled or not, wherever it comes in; and taken where forward mode is off."""
    import torch.autograd.forward_ad as fw
    y = Layer(20, 64, 96, 8, seed=1)
    W = y.wt.tensors[0]
    h, wq, wk, cos, sin, pos = _heads_inputs(20, 3, 2, 32, 16)
    q, k = (t.contiguous() for t in _split(h, 3, 2, 32))
    calls = [
        (lambda x, A, B, W: block.lora_glu(x, W, A, B, y.alpha), (y.x, y.A, y.B, W)),
        (lambda x, A, B, W, b, r: block.lora_linear_act(x, W, A, B, y.alpha, bias=b, residual=r),
         (y.x, y.A, y.B, W, y.bias, y.residual)),
        (lambda q, k, a, b, c, s: block.qk_norm_rope(q, k, a, b, c, s, pos), (q, k, wq, wk, cos, sin)),
        (lambda h, a, b, c, s: block.qkv_heads(h, 3, 2, 32, a, b, c, s, pos), (h, wq, wk, cos, sin)),
    ]
    with torch.set_grad_enabled(grad), fw.dual_level():
        for f, args in calls:
            for i, t in enumerate(args):
                dual = fw.make_dual(t, torch.ones_like(t))
                with pytest.raises(NotImplementedError, match="forward mode"):
                    f(*args[:i], dual, *args[i + 1:])
                with fw._set_fwd_grad_enabled(False):
                    f(*args[:i], dual, *args[i + 1:])
            f(*args)


def _odd(t):
    """The same values, contiguous, off every 16-byte boundary."""
    buf = torch.empty(t.numel() + 3, dtype=t.dtype, device=t.device)
    v = buf[3:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


def test_tensors_at_odd_offsets():
    """Inputs, adapters, bias, residual and norm weights off a 16-byte boundary are copied, in every
    operator; so are gradients, whose place is autograd's choice."""
    y = Layer(20, 64, 96, 8, seed=4)
    h, wq, wk, cos, sin, pos = _heads_inputs(20, 3, 2, 32, 16)
    calls = [
        (lambda x, A, B: block.lora_glu(x, y.wt, A, B, y.alpha), (y.x, y.A, y.B)),
        (lambda x, A, B, b, r: block.lora_linear_act(x, y.wt, A, B, y.alpha, bias=b, residual=r, act="silu"),
         (y.x, y.A, y.B, y.bias, y.residual)),
        (lambda x, A, B: block.lora_linear_act(x, y.wt, A, B, y.alpha), (y.x, y.A, y.B)),
        (lambda q, k, a, b: torch.cat(block.qk_norm_rope(q, k, a, b, cos, sin, pos), 1),
         (*(t.contiguous() for t in _split(h, 3, 2, 32)), wq, wk)),
        (lambda h, a, b: torch.cat(block.qkv_heads(h, 3, 2, 32, a, b, cos, sin, pos), 1), (h, wq, wk)),
    ]
    aux = torch.ones(3, dtype=torch.bfloat16, device="cuda")
    for f, args in calls:
        leaves = [t.clone().requires_grad_(True) for t in args]
        out = f(*leaves)
        up = torch.randn(out.shape, device="cuda").to(out.dtype)
        want = torch.autograd.grad(out, leaves, up)
        odd = [_odd(t).requires_grad_(True) for t in args]
        with torch.no_grad():
            assert torch.equal(f(*odd), out)
        got = f(*odd)
        assert torch.equal(got, out)
        # the gradient of `got` is a slice of the gradient of the whole, 3 elements in
        whole = torch.cat((aux, got.flatten()))
        grads = torch.autograd.grad(whole, odd, torch.cat((aux, up.flatten())))
        for a, b in zip(grads, want):
            assert torch.equal(a, b)


def test_one_token_or_one_head_with_any_stride():
    """The stride over a single token or head leads nowhere: rows of any pitch."""
    M, hq, hk, D = 6, 3, 2, 32
    h, wq, wk, cos, sin, pos = _heads_inputs(M, hq, hk, D, 16)
    n = h.shape[1]
    want = block.qkv_heads(h, hq, hk, D, wq, wk, cos, sin, pos)
    for pitch in (n + 3, n + 1):
        buf = torch.zeros(1, pitch, dtype=h.dtype, device="cuda")
        row = buf[:, :n]
        row.copy_(h[2:3])
        assert row.stride(0) == pitch
        row.requires_grad_(True)
        got = block.qkv_heads(row, hq, hk, D, wq, wk, cos, sin, pos[2:3])
        assert all(torch.equal(a, b[2:3]) for a, b in zip(got, want))
        q, k = _split(row, hq, hk, D)
        for a, b in zip(block.qk_norm_rope(q, k, wq, wk, cos, sin, pos[2:3]), want):
            assert torch.equal(a, b[2:3])
        q_out, k_out = (torch.empty_like(t) for t in (q, k))
        L.lora_qk_norm_rope_fwd(q.detach(), k.detach(), wq, wk, cos, sin, pos[2:3], q_out, k_out)
        assert torch.equal(q_out, want[0][2:3])
        d, = torch.autograd.grad(got, row, tuple(torch.ones_like(t) for t in got))
        assert d.shape == row.shape
    # one head, its own stride odd
    buf = torch.zeros(M, 3, D + 1, dtype=h.dtype, device="cuda")
    one = buf.view(M, -1)[:, :96].as_strided((M, 1, D), (96, 1000003, 1))
    assert torch.equal(block.qk_norm_rope(one, one, wq, wq, cos, sin, pos)[0],
                       block.qk_norm_rope(one.contiguous(), one.contiguous(), wq, wq, cos, sin, pos)[0])


def test_heads_that_overlap_are_copied():
    """Inputs by strides that name an element twice (windows over one row) can only be read: a copy."""
    _, wq, wk, cos, sin, pos = _heads_inputs(6, 3, 2, 32, 16)
    flat = torch.randn(8 * 32, device="cuda").to(torch.bfloat16)
    win = flat.as_strided((6, 3, 32), (32, 32, 1))
    for a, b in zip(block.qk_norm_rope(win, win[:, :2], wq, wk, cos, sin, pos),
                    block.qk_norm_rope(win.contiguous(), win[:, :2].contiguous(), wq, wk, cos, sin, pos)):
        assert torch.equal(a, b)


def test_what_is_saved_for_the_backward():
    """The frozen weight and the rotation's tables are constants of the call: no hook on saved
    tensors (save_on_cpu among them) gets them to move, and the gradients stay the same bits."""
    y = Layer(24, 64, 96, 8, "q4", seed=2)
    h, wq, wk, cos, sin, pos = _heads_inputs(24, 3, 2, 32, 16)

    def steps():
        x, A, B = (t.clone().requires_grad_(True) for t in (y.x, y.A, y.B))
        hh, a, b = (t.clone().requires_grad_(True) for t in (h, wq, wk))
        for f, leaves in ((lambda: block.lora_glu(x, y.wt, A, B, y.alpha), (x, A, B)),
                          (lambda: block.lora_linear_act(x, y.wt, A, B, y.alpha, act="silu"), (x, A, B)),
                          (lambda: torch.cat(block.qk_norm_rope(*_split(hh, 3, 2, 32), a, b, cos, sin, pos), 1), (hh, a, b)),
                          (lambda: torch.cat(block.qkv_heads(hh, 3, 2, 32, a, b, cos, sin, pos), 1), (hh, a, b))):
            out = f()
            yield from torch.autograd.grad(out, leaves, torch.ones_like(out))

    want = list(steps())
    constants = {t.data_ptr() for t in (*y.wt.tensors, cos, sin)}
    packed = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (packed.append(t.data_ptr()), t)[1], lambda t: t):
        got = list(steps())
    assert len(packed) >= 16 and not constants & set(packed)
    with torch.autograd.graph.save_on_cpu():
        moved = list(steps())
    for a, b, c in zip(want, got, moved):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_constants_changed_before_the_backward():
    """The weight, its scales or the tables changed in place between forward and backward: an error,
    as for every tensor that a backward needs."""
    y = Layer(24, 64, 96, 8, "q4", seed=2)
    h, wq, wk, cos, sin, pos = _heads_inputs(24, 3, 2, 32, 16)
    h.requires_grad_(True)
    x = y.x.clone().requires_grad_(True)
    for f, constants in ((lambda: block.lora_glu(x, y.wt, y.A, y.B, y.alpha), y.wt.tensors),
                         (lambda: block.lora_linear_act(x, y.wt, y.A, y.B, y.alpha), y.wt.tensors),
                         (lambda: block.qkv_heads(h, 3, 2, 32, wq, wk, cos, sin, pos)[0], (cos, sin, pos)),
                         (lambda: block.qk_norm_rope(*_split(h, 3, 2, 32), wq, wk, cos, sin, pos)[0], (cos, sin, pos))):
        for t in constants:
            out = f()
            t.add_(0)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                out.backward(torch.ones_like(out))
        out = f()
        out.backward(torch.ones_like(out))
        with pytest.raises(RuntimeError, match="second time"):
            out.backward(torch.ones_like(out))


def test_second_derivatives_are_errors():
    """A gradient taken with create_graph carries a node that refuses to be differentiated, also where
    the upstream gradient itself is a constant: the term is not dropped."""
    y = Layer(12, 64, 96, 8, seed=5)
    h, wq, wk, cos, sin, pos = _heads_inputs(12, 3, 2, 32, 16)
    for f, t in ((lambda x: block.lora_glu(x, y.wt, y.A, y.B, y.alpha), y.x),
                 (lambda x: block.lora_linear_act(x, y.wt, y.A, y.B, y.alpha), y.x),
                 (lambda h: block.qkv_heads(h, 3, 2, 32, wq, wk, cos, sin, pos)[0], h),
                 (lambda h: block.qk_norm_rope(*_split(h, 3, 2, 32), wq, wk, cos, sin, pos)[0], h)):
        x = t.clone().requires_grad_(True)
        out = f(x)
        want, = torch.autograd.grad(out.sum(), x, retain_graph=True)
        g, = torch.autograd.grad(out.sum(), x, create_graph=True)
        assert torch.equal(g, want)
        with pytest.raises(RuntimeError, match="twice"):
            (x.square().sum() + g.square().sum()).backward()


LOCKS = """
import sys, threading, torch
sys.path.insert(0, sys.argv[1])
from rank_linear_lora_b200 import block
def r(*s): return torch.randn(*s, device="cuda").to(torch.bfloat16)
x, W, A, B = r(200, 64), r(96, 64), r(8, 64), r(96, 8)
up = r(200, 96)
torch.cuda.memory._record_memory_history(context="all", stacks="python")
def train():
    for m in range(1, 200):
        t = x[:m].clone().requires_grad_(True)
        block.lora_linear_act(t, W, A, B, 8.0, act="silu").backward(up[:m])
def serve():
    with torch.cuda.stream(torch.cuda.Stream()), torch.no_grad():
        for m in range(1, 200):
            block.lora_linear_act(x[:m], W, A, B, 8.0)
            block.lora_glu(x[:m], W, A, B, 8.0)
ts = [threading.Thread(target=f) for f in (train, serve, train, serve)]
[t.start() for t in ts]
[t.join() for t in ts]
torch.cuda.synchronize()
print("done")
"""


def test_no_lock_is_held_over_an_allocation():
    """Threads that train and serve while every allocation records Python's stack, for which it takes
    the interpreter's lock: none waits for that lock while another waits for it (a process of its own,
    so that one that stood still would not hold up this one)."""
    r = subprocess.run([sys.executable, "-c", LOCKS, ROOT], capture_output=True, text=True, timeout=180)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), r.stderr[-2000:]


def test_waits_that_ran_out_are_reported():
    """block.check_workspaces: silent while all is well; after a bounded wait ran out in any kept
    workspace LORA_ERR_TIMEOUT, once, and the workspace is as new (zeroed whole) for the next call."""
    y = Layer(40, 64, 96, 8, seed=3)
    stream = torch.cuda.Stream()
    out = block.lora_linear_act(y.x, y.wt, y.A, y.B, y.alpha)
    with torch.cuda.stream(stream):
        block.lora_linear_act(y.x, y.wt, y.A, y.B, y.alpha)
    block.check_workspaces()
    kept = block._ops().kept_workspaces()
    mine = [w for w in kept if w.numel() == L.lora_linear_act_workspace_size(L.OP_FWD, 40, 64, 96, 8)]
    assert len(mine) >= 2
    torch.cuda.synchronize()
    for ws in mine:
        ws[256:].fill_(0x5A)
        L.lora_linear_selftest_timeout(ws, 1000)
    with pytest.raises(L.LoraError, match="block.check_workspaces") as e:
        block.check_workspaces()
    assert e.value.status == 6
    assert not any(ws.any().item() for ws in mine)
    block.check_workspaces()
    assert torch.equal(block.lora_linear_act(y.x, y.wt, y.A, y.B, y.alpha), out)
    with torch.cuda.stream(stream):
        again = block.lora_linear_act(y.x, y.wt, y.A, y.B, y.alpha)
    torch.cuda.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinities_and_nan_in_heads(inter, dtype):
    """An infinity or NaN reaches its own head alone; without the norm, its own dimension (and its
    partner in the rotation) alone, forward and backward."""
    M, hq, hk, D, rot = 9, 3, 2, 40, 16
    h, wq, wk, cos, sin, pos = _heads_inputs(M, hq, hk, D, rot, dtype=dtype)
    inf, nan = float("inf"), float("nan")
    dy = torch.randn(M, (hq + hk), D, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()

    def run(h, dy, norm):
        q, k = (t.clone().requires_grad_(True) for t in _split(h, hq, hk, D))
        out = torch.cat(block.qk_norm_rope(q, k, wq, wk, cos, sin, pos, interleaved=inter, norm=norm), 1)
        return out.detach(), torch.cat(torch.autograd.grad(out, (q, k), dy), 1)

    odd = [(1, 0, 20, inf), (2, 1, 37, -inf), (3, 2, 22, nan), (4, 3, 39, inf), (5, 4, 30, nan)]  # behind the rotation
    for norm in (False, True):
        out0, dv0 = run(h, dy, norm)
        h1, dy1 = h.clone(), dy.clone()
        for m, hd, j, v in odd:
            h1[m, hd * D + j] = v
            dy1[m, hd, j] = v
        out, _ = run(h1, dy, norm)
        _, dv = run(h, dy1, norm)
        same = torch.ones_like(out, dtype=torch.bool)
        for m, hd, j, v in odd:
            if norm:
                same[m, hd] = False
                assert out[m, hd, j].isnan()  # inf / inf
                if v == v:
                    assert not out[m, hd, [i for i in range(D) if i != j]].any()  # over an infinite root
            else:
                same[m, hd, j] = False
                w = (wq if hd < hq else wk)[j]
                for t in (out, dv):
                    assert t[m, hd, j].isnan() if v != v else t[m, hd, j] == v * w.sign()
        assert torch.equal(out[same], out0[same])
        assert torch.equal(dv[same], dv0[same])


# M, d_in, d_out, format: a few tokens with x whole and in segments, groups of 16 and of 32 rows; a
# prompt; tiles cut along K
ODD_VALUES = [
    (4, 512, 144, "bf16"), (4, 512, 4112, "q4"), (5, 576, 144, "q4"), (13, 576, 4112, "q4"), (16, 448, 272, "q4"),
    (8, 12992, 4112, "q4"), (16, 5056, 1040, "q4"), (4, 20032, 272, "q4"), (7, 576, 4112, "nf4"), (8, 12992, 272, "nf4"),
    (11, 528, 4112, "fp8"), (6, 20016, 272, "fp8"), (140, 320, 272, "bf16"), (140, 320, 272, "q4"),
    (140, 320, 272, "nf4"), (140, 336, 272, "fp8"), (40, 4160, 272, "q4"), (200, 4104, 272, "bf16"),
]


@pytest.mark.parametrize("M,d,n,fmt", ODD_VALUES, ids=["-".join(map(str, c)) for c in ODD_VALUES])
def test_infinities_nan_and_large_values(M, d, n, fmt):
    """What 64 bits give, whichever kernel runs: a token with an infinity has infinities of the
    products' signs (NaN where signs meet or a weight is zero), one with a NaN is NaN, values near the
    end of bf16 keep theirs, and the other tokens the bits that they have without these."""
    y = Layer(M, d, n, 8, fmt, seed=70 + M, alpha=8.0)
    y.A, y.B = y.A.abs(), y.B.abs()
    x = y.x.clone()
    ws = L.act_workspace(y.wt.ops()[0], M, d, n, 8)

    def run(x):
        out, p = _bf(M, n), _bf(M, n // 2)
        L.lora_linear_act_fwd(x, y.wt, y.A, y.B, None, y.residual, out, None, None, y.alpha, "none", ws)
        L.lora_glu_fwd(x, y.wt, y.A, y.B, p, None, None, y.alpha, "relu", ws)
        L.lora_linear_check(ws)
        return out, p

    plain = run(y.x)
    # E4M3 codes multiply x before the row's scale does: up to 448 times more than the result
    big = 2.0 ** 112 if fmt == "fp8" else 2.0 ** 121
    x[0, 7], x[1, d - 3], x[2, d // 2], x[3, 70] = float("inf"), float("-inf"), float("nan"), big
    if M > 4:
        x[M - 1, 11], x[M - 1, d - 11] = float("inf"), float("inf")
    out, p = run(x)
    odd = [0, 1, 2, 3] + ([M - 1] if M > 4 else [])
    rest = [i for i in range(M) if i not in odd]
    assert torch.equal(out[rest], plain[0][rest]) and torch.equal(p[rest], plain[1][rest])
    y.x = x
    h, err = y.h()
    h, err = h[odd], err[odd]
    g, u = h[:, :n // 2], h[:, n // 2:]
    a = torch.where(g < 0, torch.zeros_like(g), g)  # relu: 0 of -inf, NaN of NaN
    for name, got, want in (("out", out[odd], (h + y.residual[odd].double()).float()), ("p", p[odd], a.float() * u.float())):
        want = want.to(torch.bfloat16)  # what passes fp32 is an infinity
        if name == "p":
            # a finite g or u that is smaller than the bound of its own error has no certain sign (a weight
            # that cancels the low-rank term), and the product of the large row overflows with either
            unsure = (h.isfinite() & (h.abs() <= err))
            unsure = unsure[:, :n // 2] | unsure[:, n // 2:]
            unsure[[i for i in range(len(odd)) if odd[i] != 3]] = False
            assert unsure[3].float().mean() < 0.1
            got, want = got.masked_fill(unsure, 0), want.masked_fill(unsure, 0)
        assert torch.equal(got.isnan(), want.isnan()), name
        inf = want.isinf()
        assert torch.equal(got.isinf(), inf) and torch.equal(got[inf], want[inf]), name
    assert out[0].isposinf().any() and out[1].isneginf().any() and out[2].isnan().all() and out[3].isfinite().all()
    want, err = h[3] + y.residual[3].double(), err[3]
    assert_within("large", out[3], want, err + (HALF[torch.bfloat16] + 2 * F32) * (want.abs() + err))


@pytest.mark.parametrize("M", [4, 64])
def test_the_tail_of_gelu(M):
    """v P(v) far on the negative side, where P is small: one bf16 rounding of the value itself.  Beside
    it stand the density's exponential, whose argument v^2 / 2 <= 80 is rounded by 80 * 2^-23 in fp32, and
    __expf's own 2 + 1.2 * 80 units of 2^-23: 2^-15 together, and the fp32 rest: 2^-13 covers them."""
    d = 256
    v = -torch.linspace(1.0, 12.5, M * d, dtype=torch.float64).view(M, d).to(torch.bfloat16).cuda()
    eye = torch.eye(d, dtype=torch.bfloat16, device="cuda")
    A, B = torch.zeros(8, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(d, 8, dtype=torch.bfloat16, device="cuda")
    want, slope = act64(v.double(), "gelu")
    lim = HALF[torch.bfloat16] + 2.0 ** -13
    out = block.lora_linear_act(v, eye, A, B, 8.0, act="gelu")
    assert ((out.double() - want).abs() <= lim * want.abs()).all()
    p = block.lora_glu(v, torch.cat((eye, eye)), A, torch.cat((B, B)), 8.0, act="gelu")
    assert ((p.double() - want * v.double()).abs() <= (lim + F32) * (want * v.double()).abs()).all()
    dpre, dx = _bf(M, d), _bf(M, d)
    one, dA, dB = torch.ones_like(v), torch.empty(8, d, device="cuda"), torch.empty(d, 8, device="cuda")
    L.lora_linear_act_bwd(one, v, v, eye, A, B, None, dpre, dx, dA, dB, None, 8.0, "gelu",
                          L.act_workspace(L.OP_BWD, M, d, d, 8))
    # P + v p: its terms meet at -0.75 only
    assert ((dpre.double() - slope).abs() <= lim * slope.abs()).all()


def _act_bound(y):
    h, err = y.h()
    h, err = h + y.bias.double(), err + F32 * (h.abs() + y.bias.double().abs())
    want = h.clamp(min=0) + y.residual.double()
    return want, err + (HALF[torch.bfloat16] + 2 * F32) * (want.abs() + err)


def _glu_bound(y):
    h, err = y.h()
    n = y.n // 2
    g, u, eg, eu = h[:, :n].clamp(min=0), h[:, n:], err[:, :n], err[:, n:]
    e = eg * (u.abs() + eu) + g * eu
    return g * u, e + (HALF[torch.bfloat16] + 2 * F32) * ((g * u).abs() + e)


# M, d_in, rows of W, format: s.xa on pairs of CTAs beside the GEMM's idle SMs
PAIRS = [(1024, 4096, 4096, "bf16"), (1024, 4096, 4096, "q4"), (1000, 4104, 4080, "bf16"), (2048, 4096, 4096, "fp8")]


@pytest.mark.parametrize("M,d,n,fmt", PAIRS, ids=["-".join(map(str, c)) for c in PAIRS])
def test_rank_r_products_on_pairs_beside_the_gemm(M, d, n, fmt):
    """The GEMM starts while s.xa still runs: every element, and the same bits when x has only just been
    written by the kernel before (another projection's output, a copy)."""
    y = Layer(M, d, n, 16, fmt, seed=81)
    op = y.wt.ops()[0]
    assert L.lora_linear_act_get_plan(op, M, d, n, 16)["xa_cluster"] == 2
    ws = L.act_workspace(op, M, d, n, 16)
    out, p = _bf(M, n), _bf(M, n // 2)

    def run(x, out, p):
        L.lora_linear_act_fwd(x, y.wt, y.A, y.B, y.bias, y.residual, out, None, None, y.alpha, "relu", ws)
        L.lora_glu_fwd(x, y.wt, y.A, y.B, p, None, None, y.alpha, "relu", ws)

    run(y.x, out, p)
    L.lora_linear_check(ws)
    assert_within("out", out, *_act_bound(y))
    assert_within("p", p, *_glu_bound(y))
    # x is the output of the projection before, over a buffer that held something else
    W2 = (torch.randn(d, 64, generator=y.g) / 8).to(torch.bfloat16).cuda()
    A2, B2 = y.randn(8, 64), y.randn(d, 8)
    z = [y.randn(M, 64) for _ in range(2)]
    ws2 = L.act_workspace(L.OP_FWD, M, 64, d, 8)
    x, want = _bf(M, d), []
    for zi in z:
        L.lora_linear_act_fwd(zi, W2, A2, B2, None, None, x, None, None, 8.0, "none", ws2)
        torch.cuda.synchronize()
        o, q = _bf(M, n), _bf(M, n // 2)
        run(x.clone(), o, q)
        torch.cuda.synchronize()
        want.append((o, q))
    assert not torch.equal(want[0][0], want[1][0])
    got = []
    for i in range(20):
        L.lora_linear_act_fwd(z[i % 2], W2, A2, B2, None, None, x, None, None, 8.0, "none", ws2)
        o, q = _bf(M, n), _bf(M, n // 2)
        L.lora_linear_act_fwd(z[i % 2], W2, A2, B2, None, None, x, None, None, 8.0, "none", ws2)
        run(x, o, q)
        got.append((o, q))
    L.lora_linear_check(ws)
    for i, (o, q) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(q, want[i % 2][1]), i


def test_offsets_past_32_bits():
    """Outputs of more than 2^32 bytes and 2^31 elements: the last tokens are what they are alone (in
    the same tiles: 1024 tokens from a multiple of 1024)."""
    M, d, n = 290 * 1024, 64, 7424
    g = torch.Generator(device="cuda").manual_seed(6)

    def r(*s, k=1.0):
        return (k * torch.randn(*s, generator=g, device="cuda")).to(torch.bfloat16)

    x, W, A, B, bias = r(M, d), r(n, d, k=0.1), r(8, d, k=0.1), r(n, 8, k=0.1), r(n)
    assert M * n > 1 << 31
    res = r(1024, n).expand(290, 1024, n).reshape(M, n)
    part = slice(M - 1024, M)
    for f in (lambda x, res: block.lora_linear_act(x, W, A, B, 8.0, bias=bias, residual=res, act="silu"),
              lambda x, res: block.lora_glu(x, torch.cat((W, W)), A, torch.cat((B, B)), 8.0)):
        ends = []
        for rows in (slice(0, M), part):
            xr = x[rows].clone().requires_grad_(True)
            out = f(xr, res[rows])
            up = res[rows]
            dx, = torch.autograd.grad(out, xr, up)
            ends.append((out[-1024:].clone(), dx[-1024:].clone()))
            del out, dx, up, xr
        # other tiles may be cut along K or N: sums in another order, so half a step and fp32's own
        for a, b in zip(*ends):
            assert a.isfinite().all() and (a.double() - b.double()).abs().max() <= 2.0 ** -7 * b.double().abs().max()
    q = res.view(M, 58, 128)
    pos = torch.arange(M, device="cuda") % 64
    cos, sin = block.rope_table(64, 128, device="cuda")
    whole = block.qk_norm_rope(q, q[:, :2], None, None, cos, sin, pos)
    last = block.qk_norm_rope(q[part], q[part, :2], None, None, cos, sin, pos[part])
    assert torch.equal(whole[0][part], last[0]) and torch.equal(whole[1][part], last[1])


def test_workspaces_of_inference_mode():
    """A workspace first used under inference_mode is like any other: for training calls and the check."""
    y = Layer(44, 64, 96, 8, seed=9)
    with torch.inference_mode():
        want = block.lora_linear_act(y.x, y.wt, y.A, y.B, y.alpha).clone()
    kept = [w for w in block._ops().kept_workspaces()
            if w.numel() == L.lora_linear_act_workspace_size(L.OP_FWD, 44, 64, 96, 8)]
    assert kept and not any(w.is_inference() for w in block._ops().kept_workspaces())
    for ws in kept:
        L.lora_linear_selftest_timeout(ws, 1000)
    with pytest.raises(L.LoraError, match="TIMEOUT"):
        block.check_workspaces()
    block.check_workspaces()
    x = y.x.clone().requires_grad_(True)
    out = block.lora_linear_act(x, y.wt, y.A, y.B, y.alpha)
    out.sum().backward()
    assert torch.equal(out, want) and x.grad is not None


@pytest.mark.parametrize("reentrant", [True, False])
def test_recomputed_in_the_backward(reentrant):
    """Under checkpointing the forward runs again, in the backward's thread: the same bits."""
    from torch.utils.checkpoint import checkpoint
    y = Layer(40, 64, 128, 8, seed=12)
    cos, sin = block.rope_table(64, 16, device="cuda")
    pos = torch.arange(40, device="cuda")

    def f(x, A, B):
        p = block.lora_glu(x, y.wt, A, B, y.alpha)
        h = block.lora_linear_act(p, y.wt.tensors[0], A, B, y.alpha, act="gelu")
        return torch.cat(block.qkv_heads(h, 2, 1, 32, None, None, cos, sin, pos), 1)

    grads = []
    for again in (False, True):
        leaves = [t.clone().requires_grad_(True) for t in (y.x, y.A, y.B)]
        out = checkpoint(f, *leaves, use_reentrant=reentrant) if again else f(*leaves)
        out.square().sum().backward()
        grads.append([out.detach(), *(t.grad for t in leaves)])
    for a, b in zip(*grads):
        assert torch.equal(a, b)


def test_leading_dimensions():
    """Any leading dimensions, none among them, and one tensor in several places."""
    y = Layer(12, 64, 64, 8, seed=13)
    out = block.lora_linear_act(y.x, y.wt, y.A, y.B, y.alpha, residual=y.x)
    p = block.lora_glu(y.x, y.wt, y.A, y.B, y.alpha)
    x4 = y.x.view(2, 3, 2, 64)
    assert torch.equal(block.lora_linear_act(x4, y.wt, y.A, y.B, y.alpha, residual=x4).view(12, 64), out)
    assert torch.equal(block.lora_glu(x4, y.wt, y.A, y.B, y.alpha).view(12, 32), p)
    one = block.lora_linear_act(y.x[0], y.wt, y.A, y.B, y.alpha, residual=y.x[0])
    assert one.shape == (64,) and block.lora_glu(y.x[0], y.wt, y.A, y.B, y.alpha).shape == (32,)
    assert torch.equal(one, block.lora_linear_act(y.x[:1], y.wt, y.A, y.B, y.alpha, residual=y.x[:1])[0])
    empty = block.lora_linear_act(y.x.view(3, 4, 64)[:0], y.wt, y.A, y.B, y.alpha)
    assert empty.shape == (0, 4, 64)
    h, wq, wk, cos, sin, pos = _heads_inputs(12, 3, 2, 32, 16)
    q, k, v = block.qkv_heads(h, 3, 2, 32, wq, wk, cos, sin, pos)
    for lead in ((12,), (3, 4), (2, 3, 2)):
        for a, b in zip(block.qkv_heads(h.view(*lead, -1), 3, 2, 32, wq, wk, cos, sin, pos.view(lead)), (q, k, v)):
            assert torch.equal(a, b.view(*lead, *b.shape[1:]))
        q2, k2 = (t.unflatten(0, lead) for t in _split(h, 3, 2, 32))
        for a, b in zip(block.qk_norm_rope(q2, k2, wq, wk, cos, sin, pos.view(lead)), (q, k)):
            assert torch.equal(a, b.view(*lead, *b.shape[1:]))
    # q and k one tensor, both weights one parameter: the gradients add up
    t, w = h[:, :96].unflatten(1, (3, 32)).clone().requires_grad_(True), wq.clone().requires_grad_(True)
    a, b = block.qk_norm_rope(t, t, w, w, cos, sin, pos)
    assert torch.equal(a, b)
    both = torch.autograd.grad((a, b), (t, w), (torch.ones_like(a), torch.ones_like(b)))
    single = torch.autograd.grad(block.qk_norm_rope(t, t, w, w, cos, sin, pos)[0], (t, w), torch.ones_like(a))
    for g2, g1 in zip(both, single):
        assert torch.equal(g2, 2 * g1)


# M, d_in, rows of W, r, format
BOTH = [(1, 264, 272, 16, "bf16"), (7, 448, 528, 24, "q4"), (16, 5056, 1040, 16, "nf4"), (33, 1040, 528, 16, "bf16"),
        (200, 336, 784, 72, "fp8"), (300, 320, 528, 16, "q4"), (257, 4160, 272, 16, "nf4")]


@pytest.mark.parametrize("M,d,n,r,fmt", BOTH, ids=["-".join(map(str, c)) for c in BOTH])
def test_functions_give_the_entry_points_bits(M, d, n, r, fmt):
    """Outputs and gradients of the functions are those of the C entry points, which are compared with 64
    bits element by element; the adapters' and the bias's rounded once to their type."""
    y = Layer(M, d, n, r, fmt, seed=90 + M)
    fop, bop = y.wt.ops()

    def f32(*s):
        return torch.full(s, float("nan"), device="cuda")

    def same(got, want):
        assert all(torch.equal(a, b.to(a.dtype)) for a, b in zip(got, want))

    for act in ("none", "gelu"):
        leaves = [t.clone().requires_grad_(True) for t in (y.x, y.A, y.B, y.bias, y.residual)]
        x, A, B, bias, res = leaves
        out = block.lora_linear_act(x, y.wt, A, B, y.alpha, bias=bias, residual=res, act=act)
        up = y.randn(M, n)
        o, pre, xa = _bf(M, n), _bf(M, n), _bf(M, r)
        L.lora_linear_act_fwd(y.x, y.wt, y.A, y.B, y.bias, y.residual, o, pre, xa, y.alpha, act, L.act_workspace(fop, M, d, n, r))
        dPre, dX, dA, dB, db = _bf(M, n), _bf(M, d), f32(r, d), f32(n, r), f32(n)
        L.lora_linear_act_bwd(up, pre, y.x, y.wt, y.A, y.B, xa, dPre, dX, dA, dB, db, y.alpha, act,
                              L.act_workspace(bop, M, d, n, r))
        same((out, *torch.autograd.grad(out, leaves, up)), (o, dX, dA, dB, db, up))
        x, A, B = leaves[:3]
        p = block.lora_glu(x, y.wt, A, B, y.alpha, act=act)
        up = y.randn(M, n // 2)
        o, gu, dGU = _bf(M, n // 2), _bf(M, n), _bf(M, n)
        L.lora_glu_fwd(y.x, y.wt, y.A, y.B, o, gu, xa, y.alpha, act, L.act_workspace(fop, M, d, n, r))
        L.lora_glu_bwd(up, gu, y.x, y.wt, y.A, y.B, xa, dGU, dX, dA, dB, y.alpha, act, L.workspace(bop, M, d, n, r))
        same((p, *torch.autograd.grad(p, (x, A, B), up)), (o, dX, dA, dB))
        with torch.no_grad():  # nothing saved: the same bits
            same((block.lora_linear_act(y.x, y.wt, y.A, y.B, y.alpha, y.bias, y.residual, act),), (out,))
            same((block.lora_glu(y.x, y.wt, y.A, y.B, y.alpha, act),), (p,))
    h, wq, wk, cos, sin, pos = _heads_inputs(M, 5, 2, 64, 32)
    for inter in (False, True):
        leaves = [t.clone().requires_grad_(True) for t in (h, wq, wk)]
        outs = block.qkv_heads(leaves[0], 5, 2, 64, *leaves[1:], cos, sin, pos, eps=1e-5, interleaved=inter)
        ups = [y.randn(M, k, 64) for k in (5, 2, 2)]
        q, k = _split(h, 5, 2, 64)
        qo, ko, dh = _bf(M, 5, 64), _bf(M, 2, 64), _bf(M, 9 * 64)
        dwq, dwk = _bf(64), _bf(64)
        L.lora_qk_norm_rope_fwd(q, k, wq, wk, cos, sin, pos, qo, ko, 1e-5, inter)
        ws = torch.empty(L.lora_qk_norm_rope_workspace_size(M, 7, 64), dtype=torch.uint8, device="cuda")
        L.lora_qk_norm_rope_bwd(ups[0], ups[1], q, k, wq, wk, cos, sin, pos, *_split(dh, 5, 2, 64), dwq, dwk, ws, 1e-5, inter)
        dh[:, 7 * 64:] = ups[2].flatten(1)
        same((*outs[:2], *torch.autograd.grad(outs, leaves, ups)), (qo, ko, dh, dwq, dwk))


@pytest.mark.parametrize("M,d,n,fmt", [(1280, 2056, 4096, "bf16"), (300, 1088, 784, "q4")])
def test_plans_installed_for_the_shape(M, d, n, fmt):
    """A plan for the layer's shape steers s.xa and the last wave of the fused forwards too: any of them
    computes the same function, on workspaces of its own layout."""
    y = Layer(M, d, n, 16, fmt, seed=95)
    op = y.wt.ops()[0]
    act, glu = _act_bound(y), _glu_bound(y)
    plans = [dict(side_fwd=2), dict(side_fwd=2, splitk=[5, 0, 0, 0]), *(dict(xa_cluster=c) for c in (1, 2, 4)),
             *(dict(fwd_tail=t) for t in ((1, 2, 3) if fmt == "bf16" else (1, 2)))]
    try:
        for plan in (*plans, None):
            L.lora_linear_set_plan(M, d, n, 16, plan)
            ws = L.act_workspace(op, M, d, n, 16)
            out, p = _bf(M, n), _bf(M, n // 2)
            L.lora_linear_act_fwd(y.x, y.wt, y.A, y.B, y.bias, y.residual, out, None, None, y.alpha, "relu", ws)
            L.lora_glu_fwd(y.x, y.wt, y.A, y.B, p, None, None, y.alpha, "relu", ws)
            L.lora_linear_check(ws)
            assert_within(f"out {plan}", out, *act)
            assert_within(f"p {plan}", p, *glu)
            assert torch.equal(block.lora_linear_act(y.x, y.wt, y.A, y.B, y.alpha, y.bias, y.residual, "relu"), out)
            assert torch.equal(block.lora_glu(y.x, y.wt, y.A, y.B, y.alpha, "relu"), p)
    finally:
        L.lora_linear_set_plan(M, d, n, 16, None)
    block.check_workspaces()


def test_positions_of_any_strides():
    """Strided and expanded positions are read like contiguous ones, with and without leading dimensions."""
    h, wq, wk, cos, sin, _ = _heads_inputs(12, 3, 2, 32, 16)
    q, k = _split(h, 3, 2, 32)
    for pos in (torch.arange(24, device="cuda")[::2], torch.full((1,), 5, device="cuda").expand(12),
                torch.arange(24, device="cuda").view(12, 2)[:, 1]):
        assert not pos.is_contiguous()
        want = block.qk_norm_rope(q, k, wq, wk, cos, sin, pos.clone())
        for got in (block.qk_norm_rope(q, k, wq, wk, cos, sin, pos),
                    block.qkv_heads(h, 3, 2, 32, wq, wk, cos, sin, pos)[:2],
                    [t[0] for t in block.qk_norm_rope(q[None], k[None], wq, wk, cos, sin, pos[None])]):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
