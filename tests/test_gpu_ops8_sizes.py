"""GPU: the 8-bit dispatch of the longest row.  10 GB on the device; skipped where that much is not free."""
import pytest
import torch

import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def _room(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb * 1e9:
        pytest.skip(f"needs {gb} GB of free device memory")


def _normal(shape, seed, dtype=BF):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(seed))


def test_dispatch_of_the_longest_row():
    _room(12)
    d = (1 << 31) - 64
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(1 << 23)[:d].view(1, d)
    scales = _normal((1, mk.scale_pitch(d)), 1, F32)
    ids = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    out = {"codes": torch.zeros_like(codes), "scales": torch.zeros_like(scales)}
    mk.mk_moe_dispatch8(codes, scales, ids, None, 1, out=out)
    assert torch.equal(out["codes"], codes) and torch.equal(out["scales"], scales)
