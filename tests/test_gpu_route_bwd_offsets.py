"""Sequence bounds that the losses refuse are refused by the logits' gradient, too."""
import pytest
import torch

import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(T, E, k):
    g = torch.Generator(DEV).manual_seed(T)
    logits = torch.randn((T, E), generator=g, device=DEV)
    top = logits.topk(k, 1)
    return logits, top.indices.to(torch.int32), torch.softmax(top.values, 1), torch.randn((T, k), generator=g, device=DEV)


@pytest.mark.parametrize("T,bounds", [(100, [0, 50, 40]), (100, [1, 50, 100]), (100, [0, 50, 101]), (100, [0, -4, 100]),
                                      (100, [50, 50]), (100, [0, 60, 20, 100]), (20000, [0, 20001]),
                                      (20000, [0] + [40 * i for i in range(1, 400)] + [15959]), (1, [1, 1])])
def test_bad_bounds_are_reported_and_give_no_part(T, bounds):
    logits, ids, w, dw = _case(T, 12, 3)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    want = mk.mk_moe_route_bwd(logits, ids, topk_w=w, dweight=dw, ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK
    off = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    counts = torch.ones((len(bounds) - 1, 12), dtype=torch.int32, device=DEV)
    kw = dict(seq_offsets=off, balance_coef=0.3, z_coef=0.1, counts=counts, ws=ws)
    d = mk.mk_moe_route_bwd(logits, ids, topk_w=w, dweight=dw, **kw)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_ERR_BOUNDS
    assert torch.equal(d, want)
    assert not bool(mk.mk_moe_route_bwd(logits, ids, **kw).any())
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_ERR_BOUNDS


@pytest.mark.parametrize("bounds", [[0, 0, 0], [0, 100], [0, 0, 30, 30, 99]])
def test_good_bounds_are_not(bounds):
    logits, ids, w, dw = _case(100, 12, 3)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    off = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    counts = mk.mk_moe_balance_loss(logits, ids, seq_offsets=off)[1]
    d = mk.mk_moe_route_bwd(logits, ids, topk_w=w, dweight=dw, seq_offsets=off, balance_coef=0.3, z_coef=0.1, counts=counts,
                            ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK and bool(torch.isfinite(d).all())
