"""GPU: values of the router's losses where offsets pass 32 bits, and the norm's sum written over what was added."""
import pytest
import torch

import _ops8_ref as ref
import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def test_router_losses_past_32_bits_are_the_definition_s():
    """4.3e9 logits in three sequences (an empty one among them) and tokens behind the last.  p and lse^2 are within 2^-17
    (as in the small tests); a lane adds 1725 tokens, 2^-24 each, and partial rows and trees less than half as many: 2^-13
    of the positive sums together.  The balance loss is a sum of products of the counts, which are exact, and the means."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB of free device memory")
    T, E, k = (1 << 24) + 3, 256, 4
    logits = torch.empty((T, E), device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(6))
    logits += torch.linspace(-2, 2, E, device=DEV)  # uneven experts, so that the balance loss is not 1
    ids = torch.stack([(torch.arange(T, device=DEV) % (16 << j)) + 64 * j for j in range(3)] +
                      [torch.full((T,), 255, device=DEV)], 1).int()
    bounds = [0, (1 << 23) + 11, (1 << 23) + 11, T - 2]
    offsets = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    loss, counts, probs = mk.mk_moe_balance_loss(logits, ids, offsets)
    balance, z = 0.0, 0.0
    for s, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        if a == b:
            assert not bool(counts[s].any()) and not bool(probs[s].any())
            continue
        c = torch.bincount(ids[a:b].reshape(-1), minlength=E)
        assert torch.equal(counts[s].long(), c)
        p = torch.zeros(E, dtype=F64, device=DEV)
        for i in range(a, b, 1 << 20):
            l = logits[i:min(i + (1 << 20), b)].to(F64)
            p += torch.softmax(l, 1).sum(0)
            z += float((torch.logsumexp(l, 1) ** 2).sum())
        balance += float((c.to(F64) * E / (k * (b - a)) * p / (b - a)).sum()) / 2
    assert abs(balance - 1) > 0.1
    assert abs(float(loss[0]) / balance - 1) <= 2.0 ** -13
    assert abs(float(loss[1]) / (z / bounds[-1]) - 1) <= 2.0 ** -13


@pytest.mark.parametrize("T,d,bits8", [(1, 1, False), (700, 64, False), (700, 64, True), (2000, 129, False), (5000, 256, True),
                                       (3000, 1000, False), (900, 4095, False), (300, 16376, False), (300, 16384, True)])
def test_sum_over_the_added_tensor(T, d, bits8):
    """h may be add where both are bf16: several rows per group, rows that share 16-byte words with their neighbours."""
    g = torch.Generator(DEV).manual_seed(d)
    x = torch.empty((T, d), dtype=BF, device=DEV).normal_(generator=g)
    add = torch.empty((T, d), dtype=BF, device=DEV).normal_(generator=g)
    gamma = 1 + 0.3 * torch.randn(d, generator=g, device=DEV)
    want = mk.mk_moe_rmsnorm(x, gamma, add=add, bits8=bits8)
    assert torch.equal(want["h"], (x.float() + add.float()).to(BF))
    y, _ = ref.rmsnorm(want["h"], gamma, 1e-5)
    assert bool(((want["y"].double() - y).abs() <= (2.0 ** -8 + 2.0 ** -18) * y.abs()).all())
    kept = x.clone()
    r = mk.mk_moe_rmsnorm(x, gamma, add=add, bits8=bits8, out={"h": add})
    assert r["h"].data_ptr() == add.data_ptr() and torch.equal(x, kept)
    for name in ("h", "y", "rstd") + (("codes", "scales") if bits8 else ()):
        assert torch.equal(r[name], want[name]), name


@pytest.mark.parametrize("E", [7, 64, 256])
def test_probabilities_far_below_the_largest(E):
    """A sequence for each token, so that probs is p.  In units of 2^-24 of p, with x = logit - largest: the difference |x|,
    its product with log2 e |x| and a quarter for the constant, ex2 4; the sum of E exponentials 4 and a chain of 35; the
    reciprocal and the product 2, the mean's one."""
    g = torch.Generator(DEV).manual_seed(E)
    T = 3000
    logits = torch.randn((T, E), generator=g, device=DEV) - 86 * torch.rand((T, E), generator=g, device=DEV)
    logits += 1000 * torch.rand((T, 1), generator=g, device=DEV)
    ids = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    probs = mk.mk_moe_balance_loss(logits, ids, torch.arange(T + 1, dtype=torch.int32, device=DEV))[2].to(F64)
    l = logits.to(F64)
    p, x = torch.softmax(l, 1), l.amax(1, keepdim=True) - l
    assert float(x.max()) > 80
    assert bool(((probs - p).abs() <= (2.25 * x + 46) * 2.0 ** -24 * p + 2.0 ** -126).all())
