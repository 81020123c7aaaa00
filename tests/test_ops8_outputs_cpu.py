"""Outputs passed to the 8-bit entry points that a call does not write are refused (before any CUDA call)."""
import pytest
import torch

import dispatch_ffn_combine_gb300 as mk


def test_outputs_that_are_not_written_are_refused():
    x, gamma = torch.zeros((4, 64), dtype=torch.bfloat16), torch.ones(64)
    codes, scales = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 4))
    for out, kw in (({"h": x.clone()}, {}), ({"codes": codes}, {}), ({"scales": scales}, {}), ({"y": x}, dict(bits8=True, bf16=False)),
                    ({"codse": codes}, dict(bits8=True))):
        with pytest.raises(ValueError, match=next(iter(out))):
            mk.mk_moe_rmsnorm(x, gamma, out=out, **kw)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="x_perm"):
        mk.mk_moe_dispatch8(codes, scales, ids, None, 3, out={"x_perm": codes})
    # None stands for an output that is not passed, and h without add is x: a call's result may be passed to the next
    with pytest.raises(ValueError, match="x must be a CUDA"):
        mk.mk_moe_rmsnorm(x, gamma, out={"h": x, "codes": None, "scales": None})
