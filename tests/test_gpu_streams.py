"""GPU: calls on another stream than the current one, while the current stream
still has work on memory that was freed on the host."""
import pytest
import torch

import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
LATE = 20_000_000  # cycles, some 10 ms


def _randn(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def _tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    values = out.values() if isinstance(out, dict) else out
    return [t for t in values if t is not None]


def _training_calls():
    S, E, n, d = 133, 3, 128, 192
    off = torch.tensor([0, 33, 33, 133], dtype=torch.int32, device=DEV)
    do, x, w = _randn((S, n), 1), _randn((S, d), 2), _randn((E, n, d), 3)
    gamma, beta = torch.ones(d, device=DEV), torch.zeros(d, device=DEV)
    slot = torch.randperm(2 * S, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(S, 2).to(DEV)
    codes, scales = mk.mk_moe_ckpt8_save(x)
    _, gcodes, gscales = mk.mk_moe_swiglu_ckpt8(x, _randn((S, d), 5))
    _, mean, rstd = mk.mk_moe_layernorm(x, gamma, beta)
    return {
        "dgrad": lambda **k: mk.mk_moe_grouped_dgrad(do, off, w, **k),
        "wgrad": lambda **k: mk.mk_moe_grouped_wgrad(do, off, x, **k),
        "ckpt8_save": lambda **k: mk.mk_moe_ckpt8_save(x, **k),
        "ckpt8_dispatch": lambda **k: mk.mk_moe_ckpt8_dispatch(codes, scales, slot, **k),
        "swiglu_ckpt8": lambda **k: mk.mk_moe_swiglu_ckpt8(x, x, **k),
        "swiglu_ckpt8_bwd": lambda **k: mk.mk_moe_swiglu_ckpt8_bwd(x, gcodes, gscales, **k),
        "layernorm": lambda **k: mk.mk_moe_layernorm(x, gamma, beta, **k),
        "layernorm_bwd": lambda **k: mk.mk_moe_layernorm_bwd(x, x, gamma, mean, rstd, **k),
    }


def _check(call):
    """Memory of the call's sizes that the current stream has still to write, or to read, is not its outputs'."""
    want = [t.clone() for t in _tensors(call())]
    s = torch.cuda.Stream()
    freed = _tensors(call())
    torch.cuda.synchronize()
    torch.cuda._sleep(LATE)
    for t in freed:
        t.fill_(7)
    del freed, t
    got = _tensors(call(stream=s))
    torch.cuda.synchronize()
    for p, q in zip(want, got):
        assert torch.equal(p, q)
    # and once more with the outputs themselves: the current stream still reads them when they are freed
    torch.cuda._sleep(LATE)
    kept = [t.clone() for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got, p, q
    with torch.cuda.stream(s):
        for shape, dtype in shapes:
            torch.empty(shape, dtype=dtype, device=DEV).fill_(7)
    torch.cuda.synchronize()
    for p, q in zip(want, kept):
        assert torch.equal(p, q)


@pytest.mark.parametrize("name", ["dgrad", "wgrad", "ckpt8_save", "ckpt8_dispatch", "swiglu_ckpt8",
                                  "swiglu_ckpt8_bwd", "layernorm", "layernorm_bwd"])
def test_training_outputs_are_not_memory_in_use(name):
    _check(_training_calls()[name])


def _layer_calls():
    T, d, E, k, f = 130, 128, 4, 2, 192
    x, wg = _randn((T, d), 1), _randn((E, d), 2, d ** -0.5, torch.float32)
    w1, w3, w2 = _randn((E, f, d), 3, d ** -0.5), _randn((E, f, d), 4, d ** -0.5), _randn((E, d, f), 5, f ** -0.5)
    ids, w, _ = mk.mk_moe_route(x, wg, None, k)
    disp = mk.mk_moe_dispatch(x, ids, w, E)
    off, rows, slot, weight = (disp[n] for n in ("expert_offsets", "x_perm", "slot_row", "row_weight"))
    counts = torch.tensor([[50, 0], [30, 50]], dtype=torch.int32, device=DEV)  # of x's 130 rows
    ws = mk.alloc_workspace(T, d, E, k, f)
    mk.mk_moe_layer(x, wg, None, w1, w3, w2, k, ws=ws)
    torch.cuda.synchronize()
    return {
        "route": lambda **s: mk.mk_moe_route(x, wg, None, k, **s),
        "dispatch": lambda **s: mk.mk_moe_dispatch(x, ids, w, E, **s),
        "expert_ffn": lambda **s: mk.mk_moe_expert_ffn(rows, off, weight, w1, w3, w2, **s),
        "grouped_gemm": lambda **s: mk.mk_moe_grouped_gemm(rows, off, w1, **s),
        "dispatch_gemm": lambda **s: mk.mk_moe_dispatch_gemm(x, wg, None, w1, k, **s),
        "combine": lambda **s: mk.mk_moe_combine(rows, slot, **s),
        "layer": lambda **s: mk.mk_moe_layer(x, wg, None, w1, w3, w2, k, **s),
        "layer_routing": lambda **s: mk.mk_moe_layer_routing(ws, T, d, E, k, f, **s),
        "ep_regroup": lambda **s: mk.mk_moe_ep_regroup(x, counts, True, **s),
    }


@pytest.mark.parametrize("name", ["route", "dispatch", "expert_ffn", "grouped_gemm", "dispatch_gemm", "combine",
                                  "layer", "layer_routing", "ep_regroup"])
def test_layer_outputs_are_not_memory_in_use(name):
    _check(_layer_calls()[name])
