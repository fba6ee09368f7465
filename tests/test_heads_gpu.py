"""Norms of queries and keys with the rotation of their positions on the GPU, against 64-bit
references: types, head sizes, layouts of pairs, strides, in place, far and invalid
positions, and the gradients against the formula and against differences.

Bounds: a result is formed in fp32 and rounded once to its type (half a step).  In fp32 the
sum of squares has at most 40 additions on any path (24 in a lane, then shuffles), all of one
sign; its root, the products with the weight and the rotation add a few roundings: 40 units
of 2^-24, relative to the magnitudes that enter (|n_a| + |n_b| of the rotated pair)."""
import pytest
import torch

from block_cases import F32, HALF
from rank_linear_lora_b200 import block
from rank_linear_lora_b200 import lora_linear as L

pytestmark = pytest.mark.gpu

EPS = 1e-5
CASES = [  # M, hq, hk, D, rot, interleaved, dtype
    (1, 1, 1, 8, 8, False, torch.bfloat16),       # 8-byte vectors, one lane a head
    (1, 32, 8, 128, 128, False, torch.bfloat16),
    (8, 32, 8, 128, 128, False, torch.bfloat16),
    (7, 5, 3, 80, 40, False, torch.bfloat16),     # half a rotation of 20: 8-byte vectors
    (33, 4, 4, 96, 48, False, torch.float16),
    (300, 7, 3, 80, 48, True, torch.float32),
    (50, 3, 1, 256, 256, False, torch.float32),   # 32 lanes a head
    (50, 3, 1, 256, 128, False, torch.bfloat16),
    (5, 2, 1, 256, 8, False, torch.bfloat16),     # nearly all behind the rotation
    (9, 2, 2, 64, 0, False, torch.bfloat16),      # no rotation
    (3, 1, 1, 256, 0, False, torch.float32),
    (17, 3, 2, 72, 8, True, torch.float16),
    (64, 2, 1, 192, 96, False, torch.float32),
    (2, 70, 1, 64, 64, True, torch.bfloat16),
    (2500, 4, 2, 64, 64, False, torch.bfloat16),  # many tokens a warp in the backward
    (6000, 1, 1, 8, 8, True, torch.float32),
]
IDS = ["-".join(map(str, c)).replace("torch.", "") for c in CASES]


def _rotate(v, cos, sin, inter, sign=1):
    if cos is None:
        return v, v.abs()
    rot = 2 * cos.shape[1]
    c, s = cos[:, None], sign * sin[:, None]
    head = v[..., :rot]
    a, b = (head[..., 0::2], head[..., 1::2]) if inter else (head[..., :rot // 2], head[..., rot // 2:])
    ra, rb, m = a * c - b * s, b * c + a * s, a.abs() + b.abs()
    join = (lambda x, y: torch.stack((x, y), -1).flatten(-2)) if inter else (lambda x, y: torch.cat((x, y), -1))
    return (torch.cat((join(ra, rb), v[..., rot:]), -1), torch.cat((join(m, m), v[..., rot:].abs()), -1))


def _reference(v, w, cos, sin, inter, norm, dy=None):
    """(y, bound) or with dy (y, bound, dv, bound, dw, bound), in 64 bits."""
    half = HALF[v.dtype]
    v = v.double()
    w = torch.ones(v.shape[-1], dtype=torch.float64, device=v.device) if w is None else w.double()
    i = 1 / (v.square().mean(-1, keepdim=True) + EPS).sqrt() if norm else torch.ones_like(v[..., :1])
    e = v * i
    y, mag = _rotate(e * w, cos, sin, inter)
    out = [y, half * y.abs() + 40 * (1 + half) * F32 * mag]
    if dy is None:
        return out
    dn, dmag = _rotate(dy.double(), cos, sin, inter, -1)
    t = dn * w
    mean = (e * t).mean(-1, keepdim=True) if norm else torch.zeros_like(i)
    amean = (e * dmag * w).abs().mean(-1, keepdim=True) if norm else mean
    dv = i * (t - e * mean)
    dw = (dn * e).sum((0, 1))
    terms = v.shape[0] * v.shape[1]
    out += [dv, half * dv.abs() + 60 * (1 + half) * F32 * i * (dmag * w.abs() + e.abs() * amean),
            dw, (terms + 60) * F32 * (dmag * e.abs()).sum((0, 1))]
    return out


def _inputs(M, hq, hk, D, rot, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)

    def rnd(*s, scale=1.0):
        return (scale * torch.randn(*s, generator=g)).to(dtype).cuda()

    qkv = rnd(M, (hq + 2 * hk) * D)  # the stacked projection: rows wider than the heads
    q, k = qkv[:, :hq * D].unflatten(1, (hq, D)), qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    if M > 1:
        q[1, 0] = 0                   # a head of zeros
        q[0, 0] *= 100
    wq, wk = 1 + rnd(D, scale=0.2), 1 + rnd(D, scale=0.2)
    if rot == 0:
        return g, q, k, wq, wk, None, None, None, None, None
    cos, sin = block.rope_table(20000, rot, device="cuda")
    pos = torch.randint(0, 20000, (M,), generator=g).cuda()
    return g, q, k, wq, wk, cos, sin, pos, cos[pos].double(), sin[pos].double()


def _check(name, got, want, bound):
    over = (got.double() - want).abs() - bound
    assert not torch.isnan(over).any(), f"{name}: NaN"
    assert over.max().item() <= 0, f"{name}: {over.max().item():.3e} over its bound"


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_and_backward(case):
    M, hq, hk, D, rot, inter, dtype = case
    g, q, k, wq, wk, cos, sin, pos, c64, s64 = _inputs(*case[:5], dtype, seed=M)
    nan = lambda t: torch.full(t.shape, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    qo, ko, dq, dk = nan(q), nan(k), nan(q), nan(k)
    L.lora_qk_norm_rope_fwd(q, k, wq, wk, cos, sin, pos, qo, ko, EPS, inter)
    dqo, dko = torch.randn(q.shape, generator=g).to(dtype).cuda(), torch.randn(k.shape, generator=g).to(dtype).cuda()
    ws = torch.empty(L.lora_qk_norm_rope_workspace_size(M, hq + hk, D), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    dwq, dwk = (torch.full((D,), float("nan"), device="cuda") for _ in range(2))
    L.lora_qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, cos, sin, pos, dq, dk, dwq, dwk, ws, EPS, inter)
    torch.cuda.synchronize()
    for name, v, w, dy, got in (("q", q, wq, dqo, (qo, dq, dwq)), ("k", k, wk, dko, (ko, dk, dwk))):
        y, eb, dv, db, dw, wb = _reference(v, w, c64, s64, inter, True, dy)
        _check(name, got[0], y, eb)
        _check("d" + name, got[1], dv, db)
        _check(f"d{name}_weight", got[2], dw, wb)
    again = [torch.empty_like(t) for t in (dq, dk, dwq, dwk)]
    L.lora_qk_norm_rope_bwd(dqo, dko, q, k, wq, wk, cos, sin, pos, *again, ws, EPS, inter)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dwq, dwk)))  # a fixed order of summation


def test_parts_can_be_left_out():
    """One tensor alone, no weights, no norm, no rotation, no weight gradients."""
    M, hq, hk, D, rot = 40, 6, 2, 64, 32
    g, q, k, wq, wk, cos, sin, pos, c64, s64 = _inputs(M, hq, hk, D, rot, torch.bfloat16)
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    L.lora_qk_norm_rope_fwd(q, None, None, None, cos, sin, pos, out, None, EPS)
    _check("no weight", out, *_reference(q, None, c64, s64, False, True))
    out = torch.empty(k.shape, dtype=q.dtype, device="cuda")
    L.lora_qk_norm_rope_fwd(None, k, None, wk, cos, sin, pos, None, out, EPS, norm=False)
    _check("no norm", out, *_reference(k, wk, c64, s64, False, False))
    dy, dk = torch.randn(k.shape, generator=g).to(q.dtype).cuda(), torch.empty(k.shape, dtype=q.dtype, device="cuda")
    L.lora_qk_norm_rope_bwd(None, dy, None, k, None, wk, cos, sin, pos, None, dk, None, None, None, EPS, norm=False)
    _check("dk, no norm", dk, *_reference(k, wk, c64, s64, False, False, dy)[2:4])
    dw = torch.empty(D, device="cuda")
    ws = torch.empty(L.lora_qk_norm_rope_workspace_size(M, hk, D), dtype=torch.uint8, device="cuda")
    L.lora_qk_norm_rope_bwd(None, dy, None, k, None, wk, cos, sin, pos, None, dk, None, dw, ws, EPS, norm=False)
    _check("dk_weight, no norm", dw, *_reference(k, wk, c64, s64, False, False, dy)[4:])


def test_in_place_and_other_strides():
    """In place on the stacked projection, whose v columns and surroundings stay as they were;
    and heads outside tokens ([heads, M, D] in memory), in both directions."""
    M, hq, hk, D = 37, 4, 2, 64
    _, q, k, wq, wk, cos, sin, pos, c64, s64 = _inputs(M, hq, hk, D, 64, torch.bfloat16)
    wide = torch.full((M + 2, (hq + 2 * hk) * D + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    part = wide[1:M + 1, 32:32 + (hq + 2 * hk) * D]
    qv, kv = part[:, :hq * D].unflatten(1, (hq, D)), part[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    qv.copy_(q)
    kv.copy_(k)
    before = wide.clone()
    L.lora_qk_norm_rope_fwd(qv, kv, wq, wk, cos, sin, pos, qv, kv, EPS)
    yq, bq = _reference(q, wq, c64, s64, False, True)
    _check("q in place", qv, yq, bq)
    _check("k in place", kv, *_reference(k, wk, c64, s64, False, True))
    keep = torch.ones_like(wide, dtype=torch.bool)
    keep[1:M + 1, 32:32 + (hq + hk) * D] = False
    assert torch.equal(wide[keep], before[keep])
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(hq, M, D, dtype=q.dtype, device="cuda").transpose(0, 1)
    L.lora_qk_norm_rope_fwd(qt, None, wq, None, cos, sin, pos, out, None, EPS)
    _check("heads outside", out, yq, bq)
    dy = torch.randn(M, hq, D, device="cuda").to(q.dtype)
    dq = torch.empty(M, hq, D, dtype=q.dtype, device="cuda")
    L.lora_qk_norm_rope_bwd(dy, None, qt, None, wq, None, cos, sin, pos, dq, None, None, None, None, EPS)
    want = _reference(q, wq, c64, s64, False, True, dy)[2:4]
    _check("dq", dq, *want)
    L.lora_qk_norm_rope_bwd(dy, None, q, None, wq, None, cos, sin, pos, dy, None, None, None, None, EPS)
    _check("dq in place", dy, *want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_weight_gradients_of_the_tensors_type(dtype):
    """The fp32 sums rounded once, by the library: the bits that a cast of its fp32 outputs gives."""
    g = torch.Generator().manual_seed(12)
    q, k, dq, dk = (torch.randn(77, h, 48, generator=g).to(dtype).cuda() for h in (5, 2, 5, 2))
    w = (1 + 0.1 * torch.randn(48, generator=g)).to(dtype).cuda()
    ws = torch.empty(L.lora_qk_norm_rope_workspace_size(77, 7, 48), dtype=torch.uint8, device="cuda")
    outs = []
    for t in (torch.float32, dtype):
        dw = [torch.full((48,), 9.0, dtype=t, device="cuda") for _ in range(2)]
        L.lora_qk_norm_rope_bwd(dq, dk, q, k, w, w, None, None, None, torch.empty_like(q), torch.empty_like(k), *dw, ws, EPS)
        outs.append(dw)
    for a, b in zip(*outs):
        assert b.dtype is dtype and torch.equal(a.to(dtype), b)
    with pytest.raises(ValueError, match="dk_weight"):
        L.lora_qk_norm_rope_bwd(dq, dk, q, k, w, w, None, None, None, torch.empty_like(q), torch.empty_like(k), w.clone(),
                                torch.empty(48, dtype=torch.float64, device="cuda"), ws, EPS)


def test_positions_outside_the_table():
    """They read no table row: the token's rotated dimensions are NaN, all else is right."""
    _, q, k, wq, wk, cos, sin, pos, c64, s64 = _inputs(20, 3, 2, 64, 32, torch.bfloat16)
    pos[4], pos[11], pos[13] = -1, 20000, 1 << 40
    qo, ko = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(k.shape, dtype=q.dtype, device="cuda")
    L.lora_qk_norm_rope_fwd(q, k, wq, wk, cos, sin, pos, qo, ko, EPS)
    y, b = _reference(q, wq, c64, s64, False, True)
    bad = [4, 11, 13]
    good = [i for i in range(20) if i not in bad]
    _check("others", qo[good], y[good], b[good])
    assert qo[bad][..., :32].isnan().all() and ko[bad][..., :32].isnan().all()
    _check("unrotated", qo[bad][..., 32:], y[bad][..., 32:], b[bad][..., 32:])


def test_differences():
    """The gradients against central differences of the forward, in 32 bits: the loss is a
    fixed linear function of the outputs, a step of 2^-6 leaves a truncation of order 2^-12
    of its third derivative and a rounding of order 2^-24 / 2^-6."""
    M, hq, hk, D = 3, 2, 1, 16
    g, q, k, wq, wk, cos, sin, pos, _, _ = _inputs(M, hq, hk, D, 16, torch.float32, seed=4)
    q, k = torch.randn(q.shape, generator=g).cuda(), torch.randn(k.shape, generator=g).cuda()
    cq, ck = torch.randn(q.shape, generator=g).cuda(), torch.randn(k.shape, generator=g).cuda()

    def loss(q, k, wq, wk):
        a, b = block.qk_norm_rope(q, k, wq, wk, cos, sin, pos, eps=EPS)
        return (a.double() * cq.double()).sum().item() + (b.double() * ck.double()).sum().item()

    leaves = [t.detach().requires_grad_(True) for t in (q, k, wq, wk)]
    grads = torch.autograd.grad(block.qk_norm_rope(*leaves, cos, sin, pos, eps=EPS), leaves, (cq, ck))
    h = 2.0 ** -6
    for n in range(4):
        base = [t.detach() for t in leaves]
        for at in range(0, base[n].numel(), 7):
            vals = []
            for step in (h, -h):
                args = [t.clone() for t in base]
                args[n].view(-1)[at] += step
                vals.append(loss(*args))
            diff = (vals[0] - vals[1]) / (2 * h)
            assert abs(diff - grads[n].view(-1)[at].item()) <= 5e-3 * (1 + abs(diff)), (n, at)


def test_autograd_on_the_stacked_projection():
    """qkv_heads: q and k as the reference's, v as it is, one gradient of the stacked
    projection, gradients given as strided or expanded tensors."""
    M, hq, hk, D = 2 * 21, 4, 2, 64
    g = torch.Generator().manual_seed(8)
    h = torch.randn(2, 21, (hq + 2 * hk) * D, generator=g).to(torch.bfloat16).cuda().requires_grad_(True)
    wq = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda().requires_grad_(True)
    wk = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda().requires_grad_(True)
    cos, sin = block.rope_table(64, D, device="cuda")
    pos = torch.arange(21, device="cuda").expand(2, 21)
    q, k, v = block.qkv_heads(h, hq, hk, D, wq, wk, cos, sin, pos, eps=EPS)
    assert q.shape == (2, 21, hq, D) and v.shape == (2, 21, hk, D)
    dq = torch.randn(2, hq, 21, D, generator=g).to(torch.bfloat16).cuda().transpose(1, 2)
    dv = torch.randn(2, 21, hk, D, generator=g).to(torch.bfloat16).cuda()
    dh, dwq, dwk = torch.autograd.grad((q, k.sum(), v), (h, wq, wk), (dq, None, dv))
    h2 = h.detach().reshape(M, -1)
    c64, s64 = cos[pos.reshape(-1)].double(), sin[pos.reshape(-1)].double()
    q2, k2 = h2[:, :hq * D].unflatten(1, (hq, D)), h2[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    y, b, dx, db, dw, wb = _reference(q2, wq.detach(), c64, s64, False, True, dq.reshape(M, hq, D))
    _check("q", q.reshape(M, hq, D), y, b)
    dh2 = dh.reshape(M, -1)
    _check("dh, q", dh2[:, :hq * D].unflatten(1, (hq, D)), dx, db)
    _check("dwq", dwq, dw, wb + HALF[torch.bfloat16] * (dw.abs() + wb))
    y, b, dx, db, dw, wb = _reference(k2, wk.detach(), c64, s64, False, True, torch.ones_like(k2))
    _check("k", k.reshape(M, hk, D), y, b)
    _check("dh, k", dh2[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D)), dx, db)
    _check("dwk", dwk, dw, wb + HALF[torch.bfloat16] * (dw.abs() + wb))
    assert torch.equal(v.reshape(M, -1), h2[:, (hq + hk) * D:])
    assert torch.equal(dh2[:, (hq + hk) * D:], dv.reshape(M, -1))
    empty = block.qkv_heads(h[:0], hq, hk, D, wq, wk, cos, sin, pos[:0])
    assert [t.shape[0] for t in empty] == [0, 0, 0]


@pytest.mark.parametrize("dtype,D,rot", [(torch.bfloat16, 256, 128), (torch.float16, 72, 24), (torch.float32, 256, 64)])
def test_backward_runs_ahead_of_itself(dtype, D, rot):
    """Many units for each warp, of one step and of several, their loads in flight while others are
    computed: in place (dq over dq_out), with positions outside the table here and there, twice."""
    g = torch.Generator().manual_seed(31)
    M, hq, hk = 3000, 9, 1
    q, k, dq, dk = (torch.randn(M, h, D, generator=g).to(dtype).cuda() for h in (hq, hk, hq, hk))
    w = (1 + 0.1 * torch.randn(2, D, generator=g)).to(dtype).cuda()
    cos, sin = block.rope_table(512, rot, device="cuda")
    pos = torch.randint(0, 512, (M,), generator=g).cuda()
    bad = torch.arange(0, M, 97, device="cuda")
    good = torch.ones(M, dtype=torch.bool, device="cuda")
    good[bad] = False
    ws = torch.empty(L.lora_qk_norm_rope_workspace_size(M, hq + hk, D), dtype=torch.uint8, device="cuda")
    runs = []
    for p in (pos, pos.clone().index_fill_(0, bad, -5), pos):
        oq, ok = dq.clone(), dk.clone()
        dw = torch.empty(2, D, device="cuda")
        L.lora_qk_norm_rope_bwd(oq, ok, q, k, w[0], w[1], cos, sin, p, oq, ok, dw[0], dw[1], ws, EPS)
        runs.append((oq, ok, dw))
    for a, b in zip(runs[0], runs[2]):
        assert torch.equal(a, b)
    for a, b in zip(runs[0][:2], runs[1][:2]):
        assert torch.equal(a[good], b[good]) and b[bad].isnan().all()
    # dw_j = sum dn_j e_j: only the rotated dimensions see the angles
    assert runs[1][2][:, :rot].isnan().all() and torch.equal(runs[1][2][:, rot:], runs[0][2][:, rot:])
    c64, s64 = cos[pos].double(), sin[pos].double()
    for t, wt, dy, got, dw in ((q, w[0], dq, runs[0][0], runs[0][2][0]), (k, w[1], dk, runs[0][1], runs[0][2][1])):
        _, _, dx, db, want, wb = _reference(t, wt, c64, s64, False, True, dy)
        _check("dx", got, dx, db)
        _check("dw", dw, want, wb)
