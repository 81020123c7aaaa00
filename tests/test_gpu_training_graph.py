"""GPU: the training operators captured in CUDA graphs, the way out of their host
time on small batches: a replay on new values gives what the calls give."""
import pytest
import torch

import dispatch_ffn_combine_gb300 as mk
from dispatch_ffn_combine_gb300 import train
from dispatch_ffn_combine_gb300.workloads import CONFIGS

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


def _randn(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def _graph(f):
    """f captured after a warm-up on a side stream, and its outputs."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    return graph, out


def _cases():
    S, E, n, d = 133, 3, 128, 192
    off = torch.tensor([0, 33, 33, 133], dtype=torch.int32, device=DEV)
    long_off = torch.tensor([0, 20000], dtype=torch.int32, device=DEV)
    do, x, w = _randn((S, n), 1), _randn((S, d), 2), _randn((E, n, d), 3)
    long_do, long_x = _randn((20000, 64), 4), _randn((20000, 64), 5)
    gamma, beta = torch.ones(d, device=DEV), torch.zeros(d, device=DEV)
    slot = torch.randperm(2 * S, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(S, 2).to(DEV)

    def norm():
        y, mean, rstd = mk.mk_moe_layernorm(x, gamma, beta)
        return (y, mean, rstd, *mk.mk_moe_layernorm_bwd(x, x, gamma, mean, rstd))

    def swiglu():
        h, codes, scales = mk.mk_moe_swiglu_ckpt8(x, x)
        return (h, codes, scales, *mk.mk_moe_swiglu_ckpt8_bwd(x, codes, scales))

    def tokens():
        codes, scales = mk.mk_moe_ckpt8_save(x)
        return codes, scales, mk.mk_moe_ckpt8_dispatch(codes, scales, slot)

    return {
        "dgrad": ([do], lambda: (mk.mk_moe_grouped_dgrad(do, off, w),)),
        "wgrad": ([do, x], lambda: (mk.mk_moe_grouped_wgrad(do, off, x),)),
        "wgrad in pieces": ([long_do], lambda: (mk.mk_moe_grouped_wgrad(long_do, long_off, long_x),)),
        "norm": ([x], norm),
        "swiglu": ([x], swiglu),
        "tokens": ([x], tokens),
    }


@pytest.mark.parametrize("name", ["dgrad", "wgrad", "wgrad in pieces", "norm", "swiglu", "tokens"])
def test_operators_replayed_from_a_graph(name):
    inputs, f = _cases()[name]
    graph, out = _graph(f)
    for seed in (11, 12):
        for i, t in enumerate(inputs):
            t.copy_(_randn(t.shape, seed + i))
        want = f()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            assert torch.equal(p, q)


def test_training_step_replayed_from_a_graph():
    """A whole step.  The experts' gradients take no part in what torch multiplies (the gate's), whose library may
    choose another order under capture: they and the output are equal, the rest agrees to bf16's rounding."""
    block, x = train.make_block(CONFIGS["ragged"], seed=3)
    dout = _randn(x.shape, 2, 0.1)

    def step():
        grads = block.zero_grads()
        out, saved = train.forward(block, x)
        return out, train.backward(block, saved, dout, grads), grads

    graph, (out, dx, grads) = _graph(step)
    for seed in (21, 22):
        x.copy_(_randn(x.shape, seed))
        want, want_dx, want_grads = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for n in grads:
            if n in ("w1", "w2", "w3"):
                assert torch.equal(grads[n], want_grads[n]), n
            else:
                assert float((grads[n] - want_grads[n]).norm()) <= 2.0 ** -8 * float(want_grads[n].norm()), n
        assert float((dx.float() - want_dx.float()).norm()) <= 2.0 ** -8 * float(want_dx.float().norm())
