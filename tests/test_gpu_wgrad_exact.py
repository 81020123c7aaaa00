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


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("pieces", [False, True])
def test_wgrad_long_sum_error_in_norm(pieces, accumulate):
    """20000 rows of one expert: whole, in 27 chunks of 768 rows whose sums join in registers (the least workspace),
    and in pieces that a second kernel joins.

    A chunk is 48 MMA steps, each truncating by at most 2^-23 of the running sum, which is 2/3 of the chunk's
    sum on average (it grows with the root of the steps): 48 * 2^-23 * 2/3 = 3.8e-6 of the chunk's sum at most.
    The chunks' sums and their errors have random signs and grow alike, and the additions between them are
    rounded to nearest (2^-25 each on average): 4e-6 in norm.  One long truncated sum is at 1e-5 and more."""
    S, n, d = 20000, 256, 256
    g = torch.Generator().manual_seed(3)
    do, x = (torch.randn((S, c), generator=g).to(BF).to(DEV) for c in (n, d))
    off = _offsets([S])
    size = mk.load_library().mk_moe_grouped_wgrad_workspace_size(S, d, 1, n)
    assert size > 256
    ws = torch.empty(size if pieces else 256, dtype=torch.uint8, device=DEV)
    before = torch.randn((1, n, d), generator=g).to(DEV)
    dw = before.clone()
    mk.mk_moe_grouped_wgrad(do, off, x, dw=dw, accumulate=accumulate, ws=ws)
    want = ref.wgrad(do, off, x, 1) + (before.to(F64) if accumulate else 0)
    assert float((dw.to(F64) - want).norm() / want.norm()) <= 4e-6


@pytest.mark.parametrize("counts,n,d", [([20000], 64, 64), ([9000, 0, 3001, 1], 256, 192), ([511, 13000], 64, 256),
                                        ([767, 769, 1536, 0, 1, 2305], 320, 192)])
@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, False), (torch.float32, True), (BF, False)])
def test_wgrad_integer_sums_are_exact(counts, n, d, dtype, accumulate):
    """Operands of -2 to 2: every sum stays below 2^24 and is exact in fp32, in any order, so that a row that is lost
    or counted twice shows; whole and in pieces."""
    S, E = sum(counts), len(counts)
    assert 4 * max(counts) + 100 < 1 << 24
    off = _offsets(counts)
    g = torch.Generator().manual_seed(S)
    do, x = (torch.randint(-2, 3, (S, c), generator=g).to(BF).to(DEV) for c in (n, d))
    before = torch.randint(-100, 101, (E, n, d), generator=g).to(dtype).to(DEV)
    want = ref.wgrad(do, off, x, E) + (before.to(F64) if accumulate else 0)
    for nbytes in {256, max(256, mk.load_library().mk_moe_grouped_wgrad_workspace_size(S, d, E, n))}:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        dw = before.clone()
        mk.mk_moe_grouped_wgrad(do, off, x, dw=dw, accumulate=accumulate, ws=ws)
        assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK
        assert torch.equal(dw, want.to(dtype))
