"""The operators around the LoRA linear layer of a transformer block, with autograd.

* ``lora_glu``: gated projections of one x, act(gate) * up in the GEMM's epilogue;
* ``lora_linear_act``: a projection with bias, activation and residual in its epilogue;
* ``qk_norm_rope``: the norms of queries and keys for each head with the rotation of their
  positions (``rope_table`` makes its angles), and ``qkv_heads``, the same on the stacked
  output of the q/k/v projections;
* the modules built of them: ``LoraProjections`` (several projections of one x, each with its
  own adapter), ``LoraQKV`` and ``LoraGatedMLP``.

The projections take the frozen weight as a bf16 tensor or as a ``FrozenWeight`` of any format, and
trainable adapters A, B of the (stacked) layer; gradients flow to x, A, B, the bias and the
residual, in reverse mode, once (a second derivative, or a tensor with a tangent of forward mode,
is an error).  As ``autograd.lora_linear``: the library's kernels run, or torch's unfused
composition where the library answers LORA_ERR_UNSUPPORTED or LORA_LINEAR_FUSED=0 asks for
it (warned once); a missing library raises.  Activations, adapters, biases, norm weights and
gradients may start at any address (one off a 16-byte boundary is copied); frozen weights and the
rotation's tables start at multiples of 16 bytes.

Workspaces are kept per device, stream and shape, so calls on two streams never share one;
a call that is being captured into a CUDA graph takes a workspace of its own from the
graph's memory pool, so two graphs can replay at the same time.  The kernels' waits are bounded;
``check_workspaces`` tells whether one ran out.  To capture a backward,
capture the forward with it in the same graph (autograd runs a backward on the streams of
its forward), while no eager graph of the same leaves lives: as with torch's own operators,
autograd would accumulate on that graph's stream, and the capture raises.
"""
from __future__ import annotations

import warnings

import torch
from torch.autograd.function import once_differentiable

from . import autograd as LA
from . import lora_linear as L
from .multi import _exact_f32_product

_native = None


def _ops():
    """The native side of the operators (csrc/torch_ops.cpp): checks, workspaces, autograd."""
    global _native
    if _native is None:
        L.load_library()  # raises, with what to do, if nothing was built
        try:
            from . import _ops as native
        except ImportError as e:
            raise RuntimeError("the operators' native module is not built or does not load (run "
                               f"rank_linear_lora_b200/build.py): {e}") from e
        _native = native
    return _native


def check_workspaces():
    """Wait for the current device, then raise LoraError (LORA_ERR_TIMEOUT) if a kernel's bounded wait
    has run out in any of the operators' workspaces since the last check: the outputs of calls since
    then are not to be used.  The workspaces are zeroed again, so that later calls are right.  It sees
    the workspaces that are kept (the 64 used last); a captured call's belongs to its graph and is
    zeroed by each replay.  Synchronising: for tests and diagnostics, as lora_linear_check."""
    _ops().check_workspaces()


def _frozen(W) -> LA.FrozenWeight:
    return W if isinstance(W, LA.FrozenWeight) else LA.FrozenWeight("bf16", (W,))


def _operands(wt):
    """A FrozenWeight as the native operators take it."""
    t, kind = wt.tensors, wt.kind
    return (L.WEIGHT_FORMATS[kind], t[0], t[1] if len(t) > 1 else None,
            L._codebook(wt.codebook)[0].tolist() if kind == "nf4" else ())


def _declined(e=None):
    """Count (and warn once of) a call that takes the unfused composition; any error but
    LORA_ERR_UNSUPPORTED is raised again."""
    if e is not None and e.status != 3:
        raise e
    LA.fallback_calls += 1
    if LA.fallback_calls == 1:
        warnings.warn(f"fused LoRA operator not used ({e or 'LORA_LINEAR_FUSED=0'}); computing the unfused composition",
                      RuntimeWarning)


_TORCH_ACT = {
    "none": lambda t: t,
    "relu": torch.relu,
    "silu": torch.nn.functional.silu,
    "gelu": torch.nn.functional.gelu,
    "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh"),
}


def _rows(x):
    """x [..., d] as contiguous rows [M, d]."""
    x2 = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    return x2 if x2.is_contiguous() else x2.contiguous()


# ------------------------------------------------------------------ gated projections
def lora_glu(x, W, A, B, alpha: float, act: str = "silu"):
    """act(g) * u for [g | u] = x.W^T + (alpha / r).(x.A^T).B^T, x [..., d_in] bf16.

    W [2 d_ff, d_in] (a bf16 tensor or a FrozenWeight) holds the gate's rows and then the up
    projection's; A [r, d_in] and B [2 d_ff, r] are the stacked layer's adapters, as
    multi.SharedInputProjections lays them out (rank P r and P alpha for the call, B
    block-diagonal).  act: one of L.ACTIVATIONS."""
    wt = _frozen(W)
    code = L._act(act)
    x2 = _rows(x)
    p = None
    if LA.fused_enabled():
        try:
            p = _ops().glu(x2, A, B, alpha, code, *_operands(wt))
        except L.LoraError as e:
            _declined(e)
    else:
        _declined()
    if p is None:
        g, u = LA._unfused(x2, wt, A, B, alpha).chunk(2, dim=-1)
        p = _TORCH_ACT[act](g) * u
    return p if x.dim() == 2 else p.reshape(*x.shape[:-1], p.shape[-1])


# ------------------------------------------------------------------ projection with an epilogue
def lora_linear_act(x, W, A, B, alpha: float, bias=None, residual=None, act: str = "none"):
    """act(x.W^T + (alpha / r).(x.A^T).B^T + bias) + residual, x [..., d_in] bf16, residual
    [..., d_out], bias [d_out] (bf16), each optional.  W: a bf16 tensor [d_out, d_in] or a
    FrozenWeight.  act: one of L.ACTIVATIONS."""
    wt = _frozen(W)
    code = L._act(act)
    x2, res2 = _rows(x), residual
    if residual is not None:
        if residual.shape != (*x.shape[:-1], wt.d_out):
            raise ValueError(f"residual: expected shape {(*x.shape[:-1], wt.d_out)}, got {tuple(residual.shape)}")
        res2 = _rows(residual)
    out = None
    if LA.fused_enabled():
        try:
            out = _ops().linear_act(x2, A, B, bias, res2, alpha, code, *_operands(wt))
        except L.LoraError as e:
            _declined(e)
    else:
        _declined()
    if out is None:
        h = LA._unfused(x2, wt, A, B, alpha)
        out = _TORCH_ACT[act](h if bias is None else h + bias)
        out = out if res2 is None else out + res2
    return out if x.dim() == 2 else out.reshape(*x.shape[:-1], out.shape[-1])


# ------------------------------------------------------------------ norms of q and k with the rotation
def rope_table(n_pos: int, rot: int, theta: float = 10000.0, device=None):
    """(cos, sin) [n_pos, rot / 2] in fp32 of the angles position * theta^(-2 i / rot), formed in
    64 bits (an angle of tens of thousands of radians has no exact digits left in 32)."""
    freq = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def _unfused_heads(v, w, cos, sin, positions, eps, interleaved, norm):
    f = v.float()
    if norm:
        f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + eps)
    if w is not None:
        f = f * w.float()
    if cos is not None:
        rot = 2 * cos.shape[1]
        n = cos.shape[0]
        if n < 1 and positions.numel():
            raise ValueError("cos, sin: tables without a row")
        inside = (positions >= 0) & (positions < n)
        at = positions.clamp(0, n - 1)  # a position outside the table reads no row of it: NaN, as the kernels
        c, s = (t[at].masked_fill(~inside[:, None], float("nan"))[:, None] for t in (cos, sin))
        head = f[..., :rot]
        a, b = (head[..., 0::2], head[..., 1::2]) if interleaved else head.chunk(2, dim=-1)
        ra, rb = a * c - b * s, b * c + a * s
        turned = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
        f = torch.cat((turned, f[..., rot:]), dim=-1)
    return f.to(v.dtype)


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps: float = 1e-6,
                 interleaved: bool = False, norm: bool = True):
    """(q, k) with each head [D] over its root mean square (unless norm is False), times its
    weight, the first 2 * cos.shape[1] dimensions rotated by the token's angles.

    q [..., hq, D] and k [..., hk, D] (bf16, fp16 or fp32; column views of a stacked projection
    are read in place), weights [D] of the same type, cos and sin [n_pos, rot / 2] fp32 (see
    rope_table), positions [...] int64.  Pairs are (i, i + rot/2), or (2 i, 2 i + 1) if
    interleaved.  New tensors; gradients flow to q, k and the weights."""
    q3, k3 = (q, k) if q.dim() == 3 else (q.reshape(-1, *q.shape[-2:]), k.reshape(-1, *k.shape[-2:]))
    pos = None if positions is None else positions.reshape(-1).contiguous()
    outs = None
    if LA.fused_enabled():
        try:
            outs = _ops().qk_norm_rope(q3, k3, q_weight, k_weight, cos, sin, pos, eps, interleaved, norm)
        except L.LoraError as e:
            _declined(e)
    else:
        _declined()
    if outs is None:
        outs = (_unfused_heads(q3, q_weight, cos, sin, pos, eps, interleaved, norm),
                _unfused_heads(k3, k_weight, cos, sin, pos, eps, interleaved, norm))
    return outs if q.dim() == 3 else (outs[0].reshape(q.shape), outs[1].reshape(k.shape))


def qkv_heads(h, hq: int, hk: int, D: int, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
              eps: float = 1e-6, interleaved: bool = False, norm: bool = True):
    """(q [..., hq, D], k [..., hk, D], v [..., hk, D]) from h [..., (hq + 2 hk) D] = [q | k | v],
    the stacked output of the q/k/v projections (multi.SharedInputProjections): q and k as
    qk_norm_rope gives them, v as it is."""
    if h.shape[-1] != (hq + 2 * hk) * D:
        raise ValueError(f"h: expected {(hq + 2 * hk) * D} columns for {hq} + 2 x {hk} heads of {D}, got {h.shape[-1]}")
    h2 = _rows(h)
    pos = None if positions is None else positions.reshape(-1).contiguous()
    outs = None
    if LA.fused_enabled():
        try:
            outs = _ops().qkv_heads(h2, q_weight, k_weight, cos, sin, pos, hq, hk, D, eps, interleaved, norm)
        except L.LoraError as e:
            _declined(e)
    else:
        _declined()
    if outs is None:
        q, k, v = (t.unflatten(1, (-1, D)) for t in h2.split([hq * D, hk * D, hk * D], dim=1))
        outs = (_unfused_heads(q, q_weight, cos, sin, pos, eps, interleaved, norm),
                _unfused_heads(k, k_weight, cos, sin, pos, eps, interleaved, norm), v)
    return tuple(t.reshape(*h.shape[:-1], *t.shape[1:]) for t in outs)


# ------------------------------------------------------------------ modules
class _OwnBlocks(torch.autograd.Function):
    """B as it is; its gradient outside the blocks of the projections is zero (those entries are
    held at zero and belong to no projection)."""

    @staticmethod
    def forward(ctx, B, rows, r):
        ctx.rows, ctx.r = rows, r
        return B.view_as(B)

    @staticmethod
    @once_differentiable
    def backward(ctx, dB):
        out = torch.zeros_like(dB)
        for p, (a, b) in enumerate(ctx.rows):
            out[a:b, p * ctx.r:(p + 1) * ctx.r] = dB[a:b, p * ctx.r:(p + 1) * ctx.r]
        return out, None, None


def _layer(W, r, alpha):
    """A LoraLinear over a bf16 tensor or a FrozenWeight."""
    wt = _frozen(W)
    return LA.LoraLinear(wt.tensors[0], r, alpha) if wt.kind == "bf16" else LA.LoraLinear(r=r, alpha=alpha, frozen=wt)


class LoraProjections(torch.nn.Module):
    """P projections of one x with a frozen weight each, stacked in W [sum d_outs, d_in] (a bf16
    tensor or a FrozenWeight), and an adapter of rank r each, as
    multi.SharedInputProjections lays them out: lora_A [P r, d_in], and lora_B [sum d_outs, P r]
    block-diagonal, whose other entries stay zero.  A_p and B_p give projection p's own."""

    def __init__(self, W, d_outs, r: int = 8, alpha: float = 16.0):
        super().__init__()
        P = len(d_outs)
        self.layer = _layer(W, P * r, alpha)
        if P < 1 or sum(d_outs) != self.layer.frozen.d_out:
            raise ValueError(f"d_outs: widths that add up to the weight's {self.layer.frozen.d_out} rows, got {d_outs}")
        if not _exact_f32_product(alpha, P):
            raise ValueError(f"alpha={alpha!r}: {P}*alpha must be exact in fp32")
        self.d_outs, self.r, self.alpha = list(d_outs), r, float(alpha)
        self.layer.alpha = P * float(alpha)  # the stacked layer has rank P r: the same alpha / r
        ends = [0]
        for d in d_outs:
            ends.append(ends[-1] + d)
        self.rows = list(zip(ends, ends[1:]))

    def A_p(self, p: int):
        return self.layer.lora_A[p * self.r:(p + 1) * self.r]

    def B_p(self, p: int):
        return self.layer.lora_B[slice(*self.rows[p]), p * self.r:(p + 1) * self.r]

    def operands(self):
        """(frozen weight, A, B, alpha) of the stacked layer, for the operators above."""
        B = self.layer.lora_B
        if torch.is_grad_enabled() and B.requires_grad:
            B = _OwnBlocks.apply(B, self.rows, self.r)
        return self.layer._frozen(), self.layer.lora_A, B, self.layer.alpha

    def merged_weight(self):
        """The stacked W' = w + s.B.A in bf16 (LoraLinear.merged_weight)."""
        return self.layer.merged_weight()

    def forward(self, x):
        """[h_0 | h_1 | ...] [..., sum d_outs]."""
        return lora_linear_act(x, *self.operands())


class LoraQKV(LoraProjections):
    """The q, k and v projections of x with the norms of the heads of q and k (their weights
    q_norm and k_norm [D] are parameters; norm=False: none) and the rotation of the positions
    0 .. max_positions - 1 (its first `rot` dimensions, None: all D, 0: none; max_positions=0 leaves
    the module without a table, and then it takes no positions)."""

    def __init__(self, W, hq: int, hk: int, D: int, r: int = 8, alpha: float = 16.0, *, max_positions: int = 0,
                 rot: int = None, theta: float = 10000.0, eps: float = 1e-6, interleaved: bool = False, norm: bool = True):
        super().__init__(W, (hq * D, hk * D, hk * D), r, alpha)
        dev = self.layer.lora_A.device
        self.heads, self.eps, self.interleaved, self.norm = (hq, hk, D), eps, interleaved, norm
        for name in ("q_norm", "k_norm"):
            w = torch.nn.Parameter(torch.ones(D, dtype=torch.bfloat16, device=dev)) if norm else None
            self.register_parameter(name, w)
        if rot and not max_positions:
            raise ValueError(f"rot={rot} needs max_positions, the rows of its table")
        self.turned = rot != 0
        rot = D if rot is None else rot
        cos, sin = rope_table(max_positions, rot, theta, device=dev) if max_positions and rot else (None, None)
        self.register_buffer("cos", cos, persistent=False)
        self.register_buffer("sin", sin, persistent=False)
        self.table = max_positions, rot, theta

    def _apply(self, fn, recurse=True):
        """The angles stay in fp32 whatever type the module is converted to."""
        super()._apply(fn, recurse)
        if self.cos is not None and self.cos.dtype is not torch.float32:
            self.cos, self.sin = rope_table(*self.table, device=self.cos.device)
        return self

    def forward(self, x, positions=None):
        """(q [..., hq, D], k [..., hk, D], v [..., hk, D]); positions [...] int64."""
        if self.cos is None:
            if positions is not None and self.turned:
                raise ValueError("positions: the module has no table to rotate by (max_positions=0; rot=0 says that "
                                 "nothing is to be rotated)")
            positions = None
        elif positions is None:
            raise ValueError("positions: the tokens' positions, int64, one for each")
        return qkv_heads(super().forward(x), *self.heads, self.q_norm, self.k_norm, self.cos, self.sin, positions,
                         self.eps, self.interleaved, self.norm)


class LoraGatedMLP(torch.nn.Module):
    """down(act(gate(x)) * up(x)) + residual, an adapter of rank r on each of the three: the
    gate's and the up projection's frozen weights stacked [2 d_ff, d_in] and the down
    projection's [d_out, d_ff], each a bf16 tensor or a FrozenWeight."""

    def __init__(self, gate_up, down, r: int = 8, alpha: float = 16.0, act: str = "silu"):
        super().__init__()
        L._act(act)
        gate_up, down = _frozen(gate_up), _frozen(down)
        if gate_up.d_out != 2 * down.d_in:
            raise ValueError(f"gate and up give {gate_up.d_out // 2} values, down takes {down.d_in}")
        self.gate_up = LoraProjections(gate_up, (down.d_in, down.d_in), r, alpha)
        self.down = _layer(down, r, alpha)
        self.act = act

    def forward(self, x, residual=None):
        p = lora_glu(x, *self.gate_up.operands(), act=self.act)
        d = self.down
        return lora_linear_act(p, d._frozen(), d.lora_A, d.lora_B, d.alpha, residual=residual)
