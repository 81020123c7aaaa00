"""GPU: the grouped weight gradient where a bound on the rounding would hide a
fault: sums that are exact, errors in norm, and values below fp32's normal range."""
import numpy as np
import pytest
import torch

import _training_ref as ref
import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F64 = torch.float64
BF = torch.bfloat16


def _offsets(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)


# whole sums added to dw by the copy engine, and pieces added by the joining kernel
@pytest.mark.parametrize("counts", [[64, 0, 17], [20000]])
def test_wgrad_adds_next_to_the_normal_range(counts):
    """dw and the sums are multiples of 2^-149 around 2^-130, and a few of size 1: what is below 2^-126 may count
    as zero, three times in an element (dw, the sum, the result), so the result is within 3 * 2^-126."""
    S, E, n, d = sum(counts), len(counts), 64, 64
    off = _offsets(counts)
    g = torch.Generator().manual_seed(1)
    small = lambda shape: torch.randn(shape, generator=g) * 2.0 ** -66
    do, x = small((S, n)).to(BF).to(DEV), small((S, d)).to(BF).to(DEV)
    do[0, :4], x[0, :4] = 1.0, 1.0
    before = (torch.randn((E, n, d), generator=g, dtype=F64) * 2.0 ** -130).to(torch.float32).to(DEV)
    assert bool(before.any())
    size = mk.load_library().mk_moe_grouped_wgrad_workspace_size(S, d, E, n)
    assert (size > 256) == (S == 20000)
    dw = before.clone()
    mk.mk_moe_grouped_wgrad(do, off, x, dw=dw, accumulate=True)
    want = before.to(F64) + ref.wgrad(do, off, x, E)
    terms = ref.wgrad(do.abs(), off, x.abs(), E) + before.to(F64).abs()
    bound = 3 * 2.0 ** -126 + (max(counts) + 1) * 2.0 ** -23 * terms
    assert bool(((dw.to(F64) - want).abs() <= bound).all())
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.equal(dw[e], before[e])
