"""The operators around the layer at their edges, on the CPU: what is refused before any device work,
and the unfused compositions."""
import ctypes

import pytest
import torch

from rank_linear_lora_b200 import block
from rank_linear_lora_b200 import build as B
from rank_linear_lora_b200 import lora_linear as L

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load_library()


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("grad", [True, False], ids=["grad", "no_grad"])
def test_tangents_are_refused(lib, grad):
    """Before anything else is looked at."""
    import torch.autograd.forward_ad as fw
    x, W, A, Bm, q, h = _bf(4, 64), _bf(96, 64), _bf(8, 64), _bf(96, 8), _bf(4, 2, 16), _bf(4, 96)
    with torch.set_grad_enabled(grad), fw.dual_level():
        def dual(t):
            return fw.make_dual(t, torch.ones_like(t))

        for f in (lambda: block.lora_glu(dual(x), W, A, Bm, 8.0), lambda: block.lora_glu(x, dual(W), A, Bm, 8.0),
                  lambda: block.lora_linear_act(x, W, A, dual(Bm), 8.0),
                  lambda: block.lora_linear_act(x, W, A, Bm, 8.0, residual=dual(_bf(4, 96))),
                  lambda: block.qk_norm_rope(q, dual(q)), lambda: block.qkv_heads(dual(h), 2, 2, 16)):
            with pytest.raises(NotImplementedError, match="forward mode"):
                f()


def test_strides_over_one_token_or_head_are_not_looked_at(lib):
    """Up to the check behind the strides' (4: no workspace for the weight gradient): any stride, even a
    negative or an odd one, where there is one token or head; refused as before where there are two."""
    def bwd(M, heads, ts, hs):
        t = [ctypes.byref(L.lora_heads_t(p, ts, hs, heads)) for p in (0x7000, 0x1000, 0x5000)]
        return lib.lora_qk_norm_rope_bwd(0, t[0], None, t[1], None, None, None, P(0x2000), P(0x3000), P(0x4000), 16, t[2],
                                         None, P(0x8000), None, M, 128, 128, 0, 1, 1e-6, None, 0, None)

    assert bwd(1, 8, 1024, 128) == 4
    for ts in (0, 2057, -1, 1 << 50):
        assert bwd(1, 8, ts, 128) == 4 and bwd(1, 1, ts, ts) == 4
        assert bwd(3, 1, 1024, ts) == 4
        assert bwd(2, 8, ts, 128) in (1, 2) and bwd(1, 2, 1024, ts) in (1, 2)


def test_positions_without_a_table(monkeypatch):
    """LoraQKV does not drop positions that it has no table for; without positions, or where rot=0 says
    that nothing is rotated, it is as it was."""
    monkeypatch.setenv("LORA_LINEAR_FUSED", "0")
    W, x, pos = torch.randn(96, 32).to(torch.bfloat16), torch.randn(3, 32).to(torch.bfloat16), torch.arange(3)
    plain = block.LoraQKV(W, hq=2, hk=2, D=16, r=8)
    with pytest.raises(ValueError, match="no table"):
        plain(x, pos)
    with pytest.raises(ValueError, match="max_positions"):
        block.LoraQKV(W, hq=2, hk=2, D=16, r=8, rot=8)
    none = block.LoraQKV(W, hq=2, hk=2, D=16, r=8, rot=0, max_positions=64)
    none.load_state_dict(plain.state_dict())
    turned = block.LoraQKV(W, hq=2, hk=2, D=16, r=8, max_positions=64)
    turned.load_state_dict(plain.state_dict())
    want = plain(x)
    for got in (none(x, pos), none(x), turned(x, 0 * pos)):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not torch.equal(turned(x, pos)[0], want[0])


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
def test_unfused_positions_outside_the_table(interleaved, monkeypatch):
    """As the kernels: no row is read, the token's rotated dimensions are NaN, everything else is right.
    (Indexing with them would be an error on the CPU, a fault on a GPU, and another row for -1.)"""
    monkeypatch.setenv("LORA_LINEAR_FUSED", "0")
    g = torch.Generator().manual_seed(7)
    h = torch.randn(6, (3 + 2 * 2) * 16, generator=g)
    cos, sin = block.rope_table(32, 8)
    good, bad = torch.arange(6), torch.tensor([0, -1, 2, 32, 4, 1 << 40])
    want = block.qkv_heads(h, 3, 2, 16, None, None, cos, sin, good, interleaved=interleaved)
    got = block.qkv_heads(h, 3, 2, 16, None, None, cos, sin, bad, interleaved=interleaved)
    for a, b in zip(got[:2], want[:2]):
        assert a[[1, 3, 5], :, :8].isnan().all()
        a[[1, 3, 5], :, :8] = b[[1, 3, 5], :, :8]
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="row"):
        block.qkv_heads(h, 3, 2, 16, None, None, cos[:0], sin[:0], good)


def test_plans_of_the_fused_forwards(lib):
    """s.xa on pairs of CTAs where that leaves it the SMs that the GEMM's last round does not use, on
    fours elsewhere; tiles cut along K where there are few; nothing where the few-token kernel runs."""
    def plan(M, d_in=4096, d_out=4096, op=L.OP_FWD, r=8):
        return L.lora_linear_act_get_plan(op, M, d_in, d_out, r)

    for op in (L.OP_FWD, L.OP_FWD_Q4, L.OP_FWD_FP8, L.OP_FWD_NF4):
        assert [plan(M, op=op)["xa_cluster"] for M in (512, 1024, 2048, 4096)] == [4, 2, 2, 4]
    assert plan(256)["fwd_tail"] == 3 and plan(1024)["fwd_tail"] != 3
    assert not any(sum(v) if isinstance(v, (list, tuple)) else v for v in plan(16).values())
    assert plan(1024, r=128)["side_fwd"] == 2 and plan(1024, r=128)["splitk"][0] >= 1
    for bad in (dict(M=0), dict(M=64, op=L.OP_BWD), dict(M=64, op=8), dict(M=64, r=12), dict(M=64, d_in=96, op=L.OP_FWD_Q4)):
        with pytest.raises(L.LoraError) as e:
            plan(**bad)
        assert e.value.status == 1
