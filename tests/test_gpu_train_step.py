"""GPU: the block's training step (all training operators together).

Two references in 64 bits with the step's own routing: the step's definition,
whose backward pass uses the values that the 8-bit checkpoints stand for, and
autograd of the block's formula, from which the checkpoints may stand off."""
import pytest
import torch

import _training_ref as ref
from dispatch_ffn_combine_gb300 import train
from dispatch_ffn_combine_gb300.workloads import CONFIGS

pytestmark = pytest.mark.gpu
F64 = torch.float64
BF = torch.bfloat16


def _off(a, b):
    return float((a.to(F64) - b).norm() / b.norm().clamp(min=1e-12))


def _step(name, T, dtype):
    block, x = train.make_block(CONFIGS[name], seed=3, T=T)
    x = x.to(dtype)
    block.gamma += 0.1 * torch.randn(x.shape[1], device=x.device, generator=torch.Generator(x.device).manual_seed(1))
    dout = (0.1 * torch.randn(x.shape, device=x.device, generator=torch.Generator(x.device).manual_seed(2))).to(dtype)
    out, saved = train.forward(block, x)
    grads = block.zero_grads()
    dx = train.backward(block, saved, dout, grads)
    return block, x, dout, out, saved, grads, dx


def _definition(block, x, saved, dout):
    """The step's gradients by hand, with gate, up and tokens as their checkpoints hold them."""
    n, _, _ = ref.layernorm(x, block.gamma, block.beta, block.eps)
    n = n.to(BF)  # the layer's input is bf16
    n8 = ref.round8(n)[0].to(x.device)
    ids = saved["ids"].long()
    w = saved["w"].to(F64)
    dy = dout.to(BF).to(F64)
    g = {k: torch.zeros(v.shape, dtype=F64, device=x.device) for k, v in block.zero_grads().items()}
    dn = torch.zeros_like(n8)
    dw = torch.zeros_like(w)
    for e in range(block.w1.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        w1, w2, w3 = (getattr(block, k)[e].to(F64) for k in ("w1", "w2", "w3"))
        a = n[t].to(F64)
        gate, up = ref.round8((a @ w1.t()).to(BF))[0].to(x.device), ref.round8((a @ w3.t()).to(BF))[0].to(x.device)
        dgate, dup, hw, dw[t, j] = ref.swiglu_bwd(dy[t] @ w2, gate, up, w[t, j])
        g["w2"][e], g["w1"][e], g["w3"][e] = dy[t].t() @ hw, dgate.t() @ n8[t], dup.t() @ n8[t]
        dn.index_add_(0, t, dgate @ w1 + dup @ w3)
    dl = w * (dw - (w * dw).sum(1, keepdim=True))
    full = torch.zeros((w.shape[0], block.wg.shape[0]), dtype=F64, device=x.device).scatter_(1, ids, dl)
    g["wg"] = full.t() @ n.to(F64)
    if "bias" in g:
        g["bias"] = full.sum(0)
    dx, g["gamma"], g["beta"] = ref.layernorm_bwd(dn + full @ block.wg.to(F64), x, block.gamma, block.eps, dout)
    return dx, g


CASES = [("tiny", None, BF), ("ragged_skew", 300, torch.float32), ("edge_min", 1, BF)]


@pytest.mark.parametrize("name,T,dtype", CASES)
def test_step_matches_its_definition(name, T, dtype):
    """Every intermediate tensor is rounded to bf16 once, 2^-9 of it at most (0.2 %); at most six such roundings lie
    between dout and a gradient, and a value next to the boundary of two 8-bit codes may take the other one (a few in
    a thousand, 2^-3 apart).  2 % in norm.  The gate's gradients are differences inside a token: 5 %."""
    block, x, dout, _, saved, grads, dx = _step(name, T, dtype)
    want_dx, want = _definition(block, x, saved, dout)
    assert _off(dx, want_dx) < 2e-2
    for n, g in grads.items():
        if float(want[n].norm()) == 0:
            assert float(g.norm()) < 1e-6, n
        else:
            assert _off(g, want[n]) < (5e-2 if n in ("wg", "bias") else 2e-2), n
    again = block.zero_grads()
    assert torch.equal(train.backward(block, saved, dout, again), dx)
    train.backward(block, saved, dout, grads)  # a second micro-batch adds up
    for n in ("w1", "w2", "w3", "gamma"):
        torch.testing.assert_close(grads[n], 2 * again[n], rtol=1e-5, atol=1e-6)


def _autograd(block, x, saved, dout):
    """Gradients of <dout, x + layer(norm(x))> by autograd in 64 bits; the experts chosen are `saved`'s."""
    p = {n: getattr(block, n).to(F64).requires_grad_() for n in block.zero_grads()}
    x64 = x.to(F64).requires_grad_()
    n = torch.nn.functional.layer_norm(x64, (x.shape[1],), p["gamma"], p["beta"], block.eps)
    logits = n @ p["wg"].t() + (p["bias"] if "bias" in p else 0)
    ids = saved["ids"].long()
    w = torch.softmax(torch.gather(logits, 1, ids), 1)
    y = torch.zeros_like(n)
    for e in range(block.w1.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        a = n[t]
        h = torch.nn.functional.silu(a @ p["w1"][e].t()) * (a @ p["w3"][e].t())
        y = y.index_add(0, t, w[t, j][:, None] * (h @ p["w2"][e].t()))
    out = x64 + y
    (out * dout.to(F64)).sum().backward()
    return out.detach(), x64.grad, {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("name,T,dtype", CASES[:2])
def test_step_matches_autograd(name, T, dtype):
    """Kept in 8 bits, an activation is off by 2.6 % rms (3 bits of mantissa: 2^-4 / sqrt(12) over a binade's
    spread of sizes); gate, up and token enter each expert gradient, two of them as factors: 2.6 % sqrt(3) =
    4.5 %, and bf16 rounding of every intermediate 0.2 % each.  6 % in norm bounds the experts' and the inputs'
    gradients over many tokens.  The gate's are differences of the routing weights' gradients inside a token
    (softmax), which the same noise enters without the shared part: 12 %."""
    block, x, dout, out, saved, grads, dx = _step(name, T, dtype)
    want_out, want_dx, want = _autograd(block, x, saved, dout)
    assert _off(out, want_out) < 1e-2
    assert _off(dx, want_dx) < 6e-2
    for n, g in grads.items():
        assert _off(g, want[n]) < (0.12 if n in ("wg", "bias") else 6e-2), n


def test_training_lowers_the_loss():
    res = train.main(["--config", "ragged", "--steps", "8", "--lr", "1.0"])
    assert res["last_loss"] < 0.98 * res["first_loss"]
