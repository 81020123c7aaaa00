"""A training step of the pre-norm MoE block  out = x + layer(norm(x)).

    python -m dispatch_ffn_combine_gb300.train --config tiny --steps 20

`forward` and `backward` chain the library's forward steps and its training
operators; between them a block holds the routing tables, the norm's statistics
and 8-bit copies of the tokens and of SwiGLU's inputs, instead of the dispatched
rows and activations in 16 bits.  The weights are bf16 as in the forward layer;
their gradients are fp32 and accumulate over calls, as over micro-batches.

The norm is LayerNorm, or without a beta the root-mean-square norm.  With
coefficients for them, the step's objective includes the router's balance loss
(per sequence of the batch) and z loss.

Run as a program it fits a fixed random target with plain gradient steps on
fp32 master weights and prints the loss, and the milliseconds of a step.
"""
from __future__ import annotations

import argparse
import dataclasses
import json

import torch

from . import (mk_moe_balance_loss, mk_moe_ckpt8_dispatch, mk_moe_ckpt8_save, mk_moe_combine, mk_moe_dispatch,
               mk_moe_grouped_dgrad, mk_moe_grouped_gemm, mk_moe_grouped_wgrad, mk_moe_layernorm, mk_moe_layernorm_bwd,
               mk_moe_rmsnorm, mk_moe_rmsnorm_bwd, mk_moe_route, mk_moe_route_bwd, mk_moe_swiglu_ckpt8,
               mk_moe_swiglu_ckpt8_bwd)
from .workloads import CONFIGS, make_inputs


@dataclasses.dataclass
class MoEBlock:
    """Weights of one block: norm gamma, beta [d] fp32 (beta None: the root-mean-square norm); gate wg [E, d] fp32 (and bias [E] or None);
    experts w1, w3 [E, f, d] and w2 [E, d, f] bf16; k experts per token.  balance_coef and z_coef are the
    factors of the router's losses in the objective (0: not part of it)."""
    gamma: torch.Tensor
    beta: torch.Tensor | None
    wg: torch.Tensor
    bias: torch.Tensor | None
    w1: torch.Tensor
    w3: torch.Tensor
    w2: torch.Tensor
    k: int
    eps: float = 1e-5
    balance_coef: float = 0.0
    z_coef: float = 0.0

    def zero_grads(self) -> dict:
        """fp32 gradients of every weight, zero."""
        names = ["gamma", "beta", "wg", "w1", "w3", "w2", "bias"]
        names = [n for n in names if getattr(self, n) is not None]
        return {n: torch.zeros_like(getattr(self, n), dtype=torch.float32) for n in names}


def _norm(block: MoEBlock, x: torch.Tensor):
    """(the norm's output in bf16, mean or None, rstd)."""
    if block.beta is None:
        r = mk_moe_rmsnorm(x, block.gamma, block.eps)
        return r["y"], None, r["rstd"]
    return mk_moe_layernorm(x, block.gamma, block.beta, block.eps)


def forward(block: MoEBlock, x: torch.Tensor, seq_offsets: torch.Tensor | None = None):
    """x [T, d] (bf16 or fp32 residual stream) -> (out like x, what `backward` needs).

    seq_offsets [B + 1] int32 bounds the sequences of the router's losses (None: one of all tokens; tokens behind
    the last one have no part in them); with a coefficient that is not 0, what is saved holds them: "losses"
    [balance, z] fp32.  Their logits are the gate's product in fp32, left to torch (with its switch for tf32 on, which
    is off by default, they are rounded more than those that the router chose by).

    The layer works on bf16 whatever x is: the norm's output, gate, up, h, each expert's output and their
    sum y are rounded to it, as in the forward layer; the residual sum is in x's type."""
    E = block.w1.shape[0]
    n, mean, rstd = _norm(block, x)
    ids, w, _ = mk_moe_route(n, block.wg, block.bias, block.k)
    disp = mk_moe_dispatch(n, ids, w, E)
    off, slot_row, row_weight = disp["expert_offsets"], disp["slot_row"], disp["row_weight"]
    gate = mk_moe_grouped_gemm(disp["x_perm"], off, block.w1)
    up = mk_moe_grouped_gemm(disp["x_perm"], off, block.w3)
    h, codes, scales = mk_moe_swiglu_ckpt8(gate, up)
    y = mk_moe_combine(mk_moe_grouped_gemm(h, off, block.w2, row_weight=row_weight), slot_row)
    saved = {"x": x, "mean": mean, "rstd": rstd, "ids": ids, "w": w, "offsets": off, "slot_row": slot_row,
             "row_weight": row_weight, "act": (codes, scales), "tokens": mk_moe_ckpt8_save(n)}
    if block.balance_coef or block.z_coef:
        logits = n.float() @ block.wg.t()
        if block.bias is not None:
            logits += block.bias
        saved["losses"], counts, _ = mk_moe_balance_loss(logits, ids, seq_offsets)
        saved["gate"] = (logits, counts, seq_offsets)
    return x + y.to(x.dtype), saved


def _gate_backward(block: MoEBlock, saved: dict, drow_weight: torch.Tensor, n: torch.Tensor, grads: dict):
    """The gate's gradients from those of the routing weights; returns its part of the norm output's gradient.

    The weights are a softmax over the chosen k, so with dw[t, j] the gradient of token t's j-th weight
    dl[t, j] = w[t, j] (dw[t, j] - sum_i w[t, i] dw[t, i]) is that of its chosen logits; the others have none.
    The sums over d and T are in fp32 and left to torch.  Measured, of a whole forward and backward pass: 5.2 of
    59 ms for 32768 tokens of 7168 values and 256 experts of width 2048, 0.14 of 1.4 ms for the mid workload, 0.25 of
    1.0 ms for tiny (launches).  With the router's losses, whose gradient every logit has, both parts of dl come
    from one kernel."""
    w = saved["w"]
    if "gate" in saved:
        logits, counts, seq_offsets = saved["gate"]
        full = mk_moe_route_bwd(logits, saved["ids"], w, drow_weight, saved["slot_row"], counts, seq_offsets,
                                block.balance_coef, block.z_coef)
    else:
        dw = drow_weight[saved["slot_row"].long()]
        dl = w * (dw - (w * dw).sum(1, keepdim=True))
        full = torch.zeros((w.shape[0], block.wg.shape[0]), device=w.device).scatter_(1, saved["ids"].long(), dl)
    grads["wg"] += full.t() @ n.float()
    if block.bias is not None:
        grads["bias"] += full.sum(0)
    return full @ block.wg


def backward(block: MoEBlock, saved: dict, dout: torch.Tensor, grads: dict) -> torch.Tensor:
    """dout [T, d] in x's type -> dx; adds the weights' gradients to `grads` (see zero_grads), both of the objective
    <dout, out> + balance_coef balance + z_coef z.

    What has fewer bits than fp32, each for the types that the tensor cores and the kernels take, and for half the
    bytes: dout as it is dispatched (the residual's part of dx keeps x's type), dh, dgate, dup and the weighted
    activation, each expert's share of the norm output's gradient, their sum, and that sum with the gate's part,
    all bf16.  w1's and w3's gradients multiply the tokens, w2's the activation, as their 8-bit copies hold them;
    those copies are the larger error by far (2.6 % rms of a value against 0.2 %).  All sums are fp32."""
    off, slot_row = saved["offsets"], saved["slot_row"]
    x = saved["x"]
    # combine's gradient is the dispatch of dout; the routing weight is applied in SwiGLU's backward pass
    dP = mk_moe_dispatch(dout.to(torch.bfloat16), saved["ids"], None, block.w1.shape[0])["x_perm"]
    dh = mk_moe_grouped_dgrad(dP, off, block.w2)
    dgate, dup, hw, drow_weight = mk_moe_swiglu_ckpt8_bwd(dh, *saved["act"], row_weight=saved["row_weight"])
    mk_moe_grouped_wgrad(dP, off, hw, dw=grads["w2"], accumulate=True)
    x_perm = mk_moe_ckpt8_dispatch(*saved["tokens"], slot_row)
    mk_moe_grouped_wgrad(dgate, off, x_perm, dw=grads["w1"], accumulate=True)
    mk_moe_grouped_wgrad(dup, off, x_perm, dw=grads["w3"], accumulate=True)
    dn = mk_moe_combine(mk_moe_grouped_dgrad(dgate, off, block.w1, dup, block.w3), slot_row)
    n = _norm(block, x)[0]
    dn = (dn + _gate_backward(block, saved, drow_weight, n, grads)).to(torch.bfloat16)
    if block.beta is None:
        dx, dgamma = mk_moe_rmsnorm_bwd(dn, x, block.gamma, saved["rstd"], dres=dout)
    else:
        dx, dgamma, dbeta = mk_moe_layernorm_bwd(dn, x, block.gamma, saved["mean"], saved["rstd"], dres=dout)
        grads["beta"] += dbeta
    grads["gamma"] += dgamma
    return dx


def make_block(cfg, seed: int = 0, device="cuda", T: int | None = None, norm: str = "layer"):
    """A block and tokens x [T, d] bf16 of a named workload (see workloads); norm "layer" or "rms"."""
    inp = make_inputs(cfg, seed=seed, device=device, T=T)
    ones = torch.ones(cfg.d, device=device)
    return MoEBlock(ones, torch.zeros_like(ones) if norm == "layer" else None, inp["wg"], inp["bias"], inp["w1"], inp["w3"], inp["w2"],
                    cfg.k), inp["x"]


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--config", choices=sorted(CONFIGS), default="tiny")
    ap.add_argument("--tokens", type=int, default=None, help="override the workload's token count")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.3)
    ap.add_argument("--norm", choices=("layer", "rms"), default="layer")
    ap.add_argument("--balance", type=float, default=0.0, help="factor of the router's balance loss")
    ap.add_argument("--z", type=float, default=0.0, help="factor of the router's z loss")
    args = ap.parse_args(argv)
    block, x = make_block(CONFIGS[args.config], T=args.tokens, norm=args.norm)
    block.balance_coef, block.z_coef = args.balance, args.z
    g = torch.Generator(device=x.device).manual_seed(1)
    target = x + 0.5 * torch.randn(x.shape, generator=g, device=x.device).to(x.dtype)
    grads = block.zero_grads()
    master = {n: getattr(block, n).float() for n in grads}
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    losses, ms = [], []
    for _ in range(args.steps):
        t0.record()
        out, saved = forward(block, x)
        err = out.float() - target.float()
        backward(block, saved, (err * (2.0 / x.shape[0])).to(x.dtype), grads)
        for n, m in master.items():
            m.sub_(grads[n], alpha=args.lr)
            getattr(block, n).copy_(m)
            grads[n].zero_()
        t1.record()
        losses.append(float(err.square().sum(1).mean()))
        ms.append(t0.elapsed_time(t1))
    res = {"config": args.config, "T": x.shape[0], "steps": args.steps, "first_loss": losses[0],
           "last_loss": losses[-1], "ms_per_step": sorted(ms)[len(ms) // 2]}
    if "losses" in saved:  # of the last step
        res["balance"], res["z"] = saved["losses"].tolist()
    print(json.dumps(res))
    return res


if __name__ == "__main__":
    main()
