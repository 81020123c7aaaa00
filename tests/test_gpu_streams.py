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
