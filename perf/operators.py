"""The operators around the LoRA linear layer of a transformer block, as measured cases.

Three operators, each with its plain form (elementary torch operations in 32 bits) and the
call of this package that computes it:

  glu  gated projections of one x: h = x.W^T + s.(x.A^T).B^T with W [2 f, d] the gate rows
       and then the up rows, p = act(h[:, :f]) * h[:, f:].  The frozen W is bf16, 4-bit,
       FP8 or a 4-bit codebook's codes.  "train" adds the gradients of x, A and B.
  act  projection with an epilogue: out = act(x.W^T + s.(x.A^T).B^T + bias) + residual.
       "train" adds the gradients of x, A, B and the bias (the residual's is the output's).
  qk   norms of queries and keys: every head of every token divided by its root mean
       square, times the weight, its first `rot` dimensions rotated by the angles of the
       token's position.  "train" adds the gradients of q, k and both weights.

Scale s = alpha / r.  Everything random comes from the seed of prepare().
"""
import math

import torch

own = False

ALPHA = 32.0
EPS = 1e-6
POSITIONS = 32768  # rows of the rotation's table


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One token through the MLP's gate and up projections: generating text, one sequence.
        dict(name="glu one token", op="glu", mode="serve", M=1, d=4096, f=11008, r=32, fmt="bf16", act="silu"),
        # A few sequences generating together on the 4-bit weight of the largest MLP.
        dict(name="glu four tokens 4-bit", op="glu", mode="serve", M=4, d=8192, f=28672, r=32, fmt="q4", act="silu"),
        # A prompt of odd length on an FP8 weight of sizes no tile divides.
        dict(name="glu odd prompt fp8", op="glu", mode="serve", M=777, d=2096, f=5640, r=16, fmt="fp8", act="gelu_tanh"),
        # The MLP's first half in one fine-tuning step, 8192 tokens: forward and backward.
        dict(name="glu training step", op="glu", mode="train", M=8192, d=4096, f=11008, r=32, fmt="bf16", act="silu"),
        # One token through the MLP's down projection, added to the residual stream.
        dict(name="act one token", op="act", mode="serve", M=1, d=11008, n=4096, r=16, fmt="bf16", act="none",
             bias=False, residual=True),
        # A prompt of odd length, a codebook weight, bias and activation, odd widths.
        dict(name="act odd prompt codebook", op="act", mode="serve", M=1003, d=1088, n=2504, r=24, fmt="nf4",
             act="relu", bias=True, residual=False),
        # The down projection of a long prompt with the residual added.
        dict(name="act long prompt", op="act", mode="serve", M=8192, d=11008, n=4096, r=16, fmt="bf16", act="none",
             bias=False, residual=True),
        # An attention-sized projection with every part of the epilogue, forward and backward.
        dict(name="act training step", op="act", mode="train", M=4096, d=4096, n=4096, r=8, fmt="bf16", act="gelu",
             bias=True, residual=True),
        # Eight sequences generating together: one token of each.
        dict(name="qk eight tokens", op="qk", mode="serve", M=8, hq=32, hk=8, D=128, rot=128, interleaved=False,
             dtype="bf16"),
        # A batch of long prompts.
        dict(name="qk long prompts", op="qk", mode="serve", M=16384, hq=32, hk=8, D=128, rot=128, interleaved=False,
             dtype="bf16"),
        # The same norms in one fine-tuning step: forward and backward.
        dict(name="qk training step", op="qk", mode="train", M=8192, hq=32, hk=8, D=128, rot=128, interleaved=False,
             dtype="bf16"),
        # Odd head counts and sizes, a part of the head rotated, pairs next to each other, 32 bits.
        dict(name="qk odd heads fp32", op="qk", mode="train", M=1999, hq=7, hk=3, D=80, rot=48, interleaved=True,
             dtype="fp32"),
    ]


LARGEST = 8192 * 4096 * 2 * 11008  # products of the largest listed projection


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glu", "act", "qk"])
    mode = rng.choice(["serve", "serve", "train"])
    if op == "qk":
        hk = rng.randint(1, 16)
        D = rng.choice([64, 80, 96, 128, 192, 256])
        hq = hk * rng.randint(1, 8) if rng.random() < 0.7 else rng.randint(1, 64)
        M = _log(rng, 1, 16384)
        M = max(1, min(M, 16384 * 40 * 128 // ((hq + hk) * D)))
        return dict(op=op, mode=mode, M=M, hq=hq, hk=hk, D=D, rot=rng.choice([D, D, D // 2 // 8 * 8]),
                    interleaved=rng.random() < 0.3, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    fmt = rng.choice(["bf16", "bf16", "q4", "fp8", "nf4"])
    unit = {"bf16": 8, "fp8": 16, "q4": 64, "nf4": 64}[fmt]
    d = max(1, _log(rng, 256, 8192) // unit) * unit
    wide = max(1, _log(rng, 256, 12288) // 8) * 8
    M = max(1, min(_log(rng, 1, 8192), LARGEST // (2 * d * wide)))
    case = dict(op=op, mode=mode, M=M, d=d, r=rng.choice([8, 16, 24, 32, 64]), fmt=fmt,
                act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]))
    if op == "glu":
        return dict(case, f=wide)
    return dict(case, n=wide, act=rng.choice(["none", "none", case["act"]]), bias=rng.random() < 0.5,
                residual=rng.random() < 0.6)


# ------------------------------------------------------------------ inputs
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _weight(g, fmt, n, d):
    """A frozen weight of standard deviation 1 / sqrt(d), as its format stores it."""
    if fmt == "bf16":
        return (torch.randn(n, d, generator=g, device="cuda") / d ** 0.5).to(torch.bfloat16),
    if fmt == "fp8":  # E4M3 codes of N(0, 64^2) values, one scale a row
        q = (torch.randn(n, d, generator=g, device="cuda") * 64).clamp_(-448, 448).to(torch.float8_e4m3fn)
        sc = (1 + 0.2 * torch.rand(n, generator=g, device="cuda")) / (64 * d ** 0.5)
        return q.view(torch.uint8), sc.to(torch.bfloat16)
    spread = 4.3 / 7 if fmt == "q4" else 0.6  # standard deviation of the decoded codes
    lo = torch.randint(1 if fmt == "q4" else 0, 16, (n, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    hi = torch.randint(1 if fmt == "q4" else 0, 16, (n, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    sc = (1 + 0.2 * torch.rand(n, d // 64, generator=g, device="cuda")) / (spread * d ** 0.5)
    return lo | (hi << 4), sc.to(torch.bfloat16)


# 16 increasing values from -1 to 1 with a zero, denser near it
CODEBOOK = [-1.0, -0.7, -0.52, -0.39, -0.28, -0.18, -0.09, 0.0, 0.08, 0.16, 0.25, 0.34, 0.44, 0.56, 0.72, 1.0]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (std * torch.randn(*shape, generator=g, device="cuda")).to(dtype)

    s = dict(case)
    M = case["M"]
    if case["op"] == "qk":
        dt, hq, hk, D, rot = DTYPES[case["dtype"]], case["hq"], case["hk"], case["D"], case["rot"]
        # q and k are the first columns of the stacked projection [q | k | v]
        qkv = normal(M, (hq + 2 * hk) * D, dtype=dt)
        s["q"] = qkv[:, :hq * D].unflatten(1, (hq, D))
        s["k"] = qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
        s["wq"], s["wk"] = 1 + normal(D, std=0.1, dtype=dt), 1 + normal(D, std=0.1, dtype=dt)
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = torch.arange(POSITIONS, dtype=torch.float64, device="cuda")[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        # every token of a prompt in order from some place on; generated ones anywhere
        if M < 64:
            s["pos"] = torch.randint(0, POSITIONS, (M,), generator=g, device="cuda")
        else:
            start = torch.randint(0, POSITIONS - M + 1, (1,), generator=g, device="cuda")
            s["pos"] = torch.arange(M, device="cuda") + start
        if case["mode"] == "train":
            s["dq"], s["dk"] = normal(M, hq, D, dtype=dt), normal(M, hk, D, dtype=dt)
            for name in ("q", "k", "wq", "wk"):
                s[name] = s[name].detach().requires_grad_(True)
        return s
    d, r = case["d"], case["r"]
    n = 2 * case["f"] if case["op"] == "glu" else case["n"]
    wide = case["f"] if case["op"] == "glu" else n
    s["x"] = normal(M, d)
    s["W"] = _weight(g, case["fmt"], n, d)
    s["A"] = ((2 * torch.rand(r, d, generator=g, device="cuda") - 1) / d ** 0.5).to(torch.bfloat16)
    s["B"] = normal(n, r, std=0.02)
    if case.get("bias"):
        s["b"] = normal(n, std=0.5)
    if case.get("residual"):
        s["res"] = normal(M, n)
    if case["mode"] == "train":
        s["dout"] = normal(M, wide)
        for name in ("x", "A", "B", "b"):
            if name in s:
                s[name] = s[name].detach().requires_grad_(True)
    return s


# ------------------------------------------------------------------ plain forms
def _decoded(W, fmt):
    """The frozen weight in 32 bits."""
    if fmt == "bf16":
        return W[0].float()
    if fmt == "fp8":
        return W[0].view(torch.float8_e4m3fn).float() * W[1].float()[:, None]
    q = torch.stack((W[0] & 15, W[0] >> 4), dim=-1).flatten(1)
    table = (torch.arange(16, device=q.device) - 8) / 7.0 if fmt == "q4" else torch.tensor(CODEBOOK, device=q.device)
    return (table[q.int()].unflatten(1, (-1, 64)) * W[1].float()[:, :, None]).flatten(1)


def _act(h, act):
    """(act(h), its derivative), both in h's precision."""
    if act == "none":
        return h, torch.ones_like(h)
    if act == "relu":
        return h.clamp(min=0), (h > 0).to(h.dtype)
    if act == "silu":
        sg = torch.sigmoid(h)
        return h * sg, sg * (1 + h * (1 - sg))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(h * 0.5 ** 0.5))
        return h * cdf, cdf + h * torch.exp(-0.5 * h * h) * (2 * math.pi) ** -0.5
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (h + 0.044715 * h ** 3))
    return 0.5 * h * (1 + t), 0.5 * (1 + t) + 0.5 * h * (1 - t * t) * c * (1 + 3 * 0.044715 * h * h)


def _plain_projection(s):
    x, W, A, B = s["x"].detach().float(), _decoded(s["W"], s["fmt"]), s["A"].detach().float(), s["B"].detach().float()
    scale = ALPHA / s["r"]
    xa = scale * (x @ A.t())
    h = x @ W.t() + xa @ B.t()
    bf = torch.bfloat16
    if s["op"] == "glu":
        gate, up = h[:, :s["f"]], h[:, s["f"]:]
        a, da = _act(gate, s["act"])
        out = (a * up).to(bf)
        if s["mode"] == "serve":
            return out
        do = s["dout"].float()
        dh = torch.cat((do * up * da, do * a), dim=1)
    else:
        if "b" in s:
            h = h + s["b"].detach().float()
        a, da = _act(h, s["act"])
        out = (a + s["res"].float() if "res" in s else a).to(bf)
        if s["mode"] == "serve":
            return out
        dh = s["dout"].float() * da
    ga = scale * (dh @ B)
    dx, dA, dB = dh @ W + ga @ A, ga.t() @ x, dh.t() @ xa
    grads = [dx.to(bf), dA.to(bf), dB.to(bf)]
    return (out, *grads, dh.sum(0).to(bf)) if "b" in s else (out, *grads)


def _rotated(v, cos, sin, interleaved, back=False):
    """The first 2 * cos.shape[-1] dimensions of v [M, H, D] rotated (back: by the negative angles)."""
    half = cos.shape[-1]
    sin = -sin if back else sin
    cos, sin = cos[:, None, :], sin[:, None, :]
    head, rest = v[..., :2 * half], v[..., 2 * half:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _plain_heads(v, w, cos, sin, interleaved, dy=None):
    """One of q and k: the output, or with dy the gradients of v and w too."""
    dt = v.dtype
    v, w = v.detach().float(), w.detach().float()
    inv = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    unit = v * inv
    y = _rotated(unit * w, cos, sin, interleaved).to(dt)
    if dy is None:
        return y
    dn = _rotated(dy.float(), cos, sin, interleaved, back=True)
    dw = (dn * unit).sum((0, 1))
    du = dn * w
    return y, (inv * (du - unit * (du * unit).mean(-1, keepdim=True))).to(dt), dw.to(dt)


def _plain_qk(s):
    cos, sin = s["cos"][s["pos"]], s["sin"][s["pos"]]
    i = s["interleaved"]
    if s["mode"] == "serve":
        return _plain_heads(s["q"], s["wq"], cos, sin, i), _plain_heads(s["k"], s["wk"], cos, sin, i)
    q, dq, dwq = _plain_heads(s["q"], s["wq"], cos, sin, i, s["dq"])
    k, dk, dwk = _plain_heads(s["k"], s["wk"], cos, sin, i, s["dk"])
    return q, k, dq, dk, dwq, dwk


# ------------------------------------------------------------------ this package's calls
def _own(s):
    from rank_linear_lora_b200 import autograd, block
    train = s["mode"] == "train"
    if s["op"] == "qk":
        with torch.set_grad_enabled(train):
            q, k = block.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], eps=EPS,
                                      interleaved=s["interleaved"])
        if not train:
            return q, k
        return (q, k, *torch.autograd.grad((q, k), (s["q"], s["k"], s["wq"], s["wk"]), (s["dq"], s["dk"])))
    W = autograd.FrozenWeight(s["fmt"], s["W"], codebook=CODEBOOK if s["fmt"] == "nf4" else None)
    with torch.set_grad_enabled(train):
        if s["op"] == "glu":
            out = block.lora_glu(s["x"], W, s["A"], s["B"], ALPHA, act=s["act"])
        else:
            out = block.lora_linear_act(s["x"], W, s["A"], s["B"], ALPHA, bias=s.get("b"), residual=s.get("res"),
                                        act=s["act"])
    if not train:
        return out
    leaves = [s[name] for name in ("x", "A", "B", "b") if name in s]
    return (out.detach(), *torch.autograd.grad(out, leaves, s["dout"]))


def run(state):
    if own:
        return _own(state)
    return _plain_qk(state) if state["op"] == "qk" else _plain_projection(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    M, train = case["M"], case["mode"] == "train"
    if case["op"] == "qk":
        e, H, D = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]], case["hq"] + case["hk"], case["D"]
        table = M * (8 + case["rot"] * 4)
        passes = 4 if train else 2  # in and out; dy in and dx out
        return {"bytes": passes * M * H * D * e + table + (4 if train else 2) * D * e,
                "flops": M * H * D * (20 if train else 8)}
    d, r = case["d"], case["r"]
    n = 2 * case["f"] if case["op"] == "glu" else case["n"]
    wide = case["f"] if case["op"] == "glu" else n
    weight = n * d * {"bf16": 2, "fp8": 1, "q4": 0.5, "nf4": 0.5}[case["fmt"]]
    weight += {"bf16": 0, "fp8": 2 * n, "q4": n * d / 32, "nf4": n * d / 32}[case["fmt"]]
    extra = 2 * n * bool(case.get("bias")) + 2 * M * n * bool(case.get("residual"))
    data = weight + 2 * (M * d + r * d + n * r) + 2 * M * wide + extra
    flops = 2 * M * n * d + 2 * M * r * (n + d)
    if train:
        data += 2 * M * wide + 2 * (M * d + r * d + n * r) + 2 * n * bool(case.get("bias"))
        flops += 2 * M * n * d + 4 * M * r * (n + d)
    return {"bytes": int(data), "flops": int(flops)}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_weight(s):
    fmt, W = s["fmt"], s["W"]
    if fmt == "bf16":
        return W[0].double()
    if fmt == "fp8":
        c = W[0].long()
        e, m = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m / 8 * 2.0 ** -6)
        return torch.where(c >= 128, -mag, mag) * W[1].double().unsqueeze(1)
    n, half = W[0].shape
    w = torch.empty(n, 2 * half, dtype=torch.float64, device=W[0].device)
    for odd in (0, 1):
        code = (W[0].int() >> (4 * odd)) & 15
        w[:, odd::2] = (code.double() - 8) / 7 if fmt == "q4" else W[0].new_tensor(CODEBOOK, dtype=torch.float64)[code]
    return w * W[1].double().repeat_interleave(64, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    F = torch.nn.functional
    train = case["mode"] == "train"
    with torch.enable_grad():
        if case["op"] == "qk":
            outs, leaves, ups = [], [], []
            turn = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"]].unsqueeze(1)
            for v, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
                v, w = v.detach().double().requires_grad_(train), w.detach().double().requires_grad_(train)
                y = w * v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)
                rot = case["rot"]
                pairs = y[..., :rot].unflatten(-1, (rot // 2, 2) if case["interleaved"] else (2, rot // 2))
                pairs = pairs if case["interleaved"] else pairs.transpose(-1, -2)
                z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
                z = z if case["interleaved"] else z.transpose(-1, -2)
                outs.append(torch.cat((z.flatten(-2), y[..., rot:]), dim=-1))
                leaves += [v, w]
                ups.append(dy)
            if not train:
                return tuple(outs)
            dq, dwq, dk, dwk = torch.autograd.grad(outs, leaves, [u.double() for u in ups])
            return outs[0].detach(), outs[1].detach(), dq, dk, dwq, dwk
        leaf = {k: s[k].detach().double().requires_grad_(train) for k in ("x", "A", "B", "b") if k in s}
        W = _exact_weight(s)
        h = F.linear(leaf["x"], W) + (ALPHA / case["r"]) * F.linear(F.linear(leaf["x"], leaf["A"]), leaf["B"])
        if "b" in leaf:
            h = h + leaf["b"]
        f = {"none": lambda t: t, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
             "gelu_tanh": lambda t: F.gelu(t, approximate="tanh")}[case["act"]]
        if case["op"] == "glu":
            gate, up = h.chunk(2, dim=1)
            out = f(gate) * up
        else:
            out = f(h) + (s["res"].double() if "res" in s else 0)
        if not train:
            return out
        return (out.detach(), *torch.autograd.grad(out, list(leaf.values()), s["dout"].double()))
