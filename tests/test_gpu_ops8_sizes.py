"""GPU: the 8-bit path on rows of more than 2^31 values in all, and on the longest row.  5 to 15 GB on the device; skipped
where that much is not free."""
import pytest
import torch

import dispatch_ffn_combine_gb300 as mk
from dispatch_ffn_combine_gb300 import block8

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def _room(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb * 1e9:
        pytest.skip(f"needs {gb} GB of free device memory")


def _normal(shape, seed, dtype=BF):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(seed))


def _offsets(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def test_dispatch_of_the_longest_row():
    _room(12)
    d = (1 << 31) - 64
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(1 << 23)[:d].view(1, d)
    scales = _normal((1, mk.scale_pitch(d)), 1, F32)
    ids = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    out = {"codes": torch.zeros_like(codes), "scales": torch.zeros_like(scales)}
    mk.mk_moe_dispatch8(codes, scales, ids, None, 1, out=out)
    assert torch.equal(out["codes"], codes) and torch.equal(out["scales"], scales)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_product_of_more_than_2_31_row_values(dtype):
    """A row's result does not depend on where it lies: parts of a large call are those of a small one, bit for bit."""
    _room(20)
    S, d, E, n = 330_001, 7168, 3, 320
    codes, scales = mk.mk_moe_quant8_rows(_normal((S, d), 3))
    w = mk.mk_moe_quant8_weights(_normal((E, n, d), 5))
    off = [0, 299_700, 299_700, S]
    out = mk.mk_moe_grouped_gemm8(codes, scales, _offsets(off), *w, dtype=dtype)
    for e in (0, 2):
        one = w[0][e:e + 1], w[1][e:e + 1]
        for a, b in ((off[e], off[e] + 300), (299_500, 299_700) if e == 0 else (299_700, 300_100), (off[e + 1] - 300, off[e + 1])):
            part = mk.mk_moe_grouped_gemm8(codes[a:b], scales[a:b], _offsets([0, b - a]), *one, dtype=dtype)
            assert torch.equal(part, out[a:b]), (e, a)


def test_block_of_more_tokens_than_37449():
    """Eight rows of 7168 values for each of 40003 tokens; each token's output is that of a small batch."""
    _room(20)
    T, d, E, f, k = 40_003, 7168, 8, 128, 8
    w13 = mk.mk_moe_quant8_weights(_normal((E, 2 * f, d), 1) * d ** -0.5)
    w2 = mk.mk_moe_quant8_weights(_normal((E, d, f), 2) * f ** -0.5)
    block = block8.Block8(torch.ones(d, device=DEV), _normal((E, d), 3, F32) * d ** -0.5, None, w13, w2, k)
    x, add = _normal((T, d), 4), _normal((T, d), 5)
    h, y = block8.forward(block, x, add)
    for a, b in ((0, 200), (37_400, 37_500), (T - 203, T)):
        ph, py = block8.forward(block, x[a:b], add[a:b])
        assert torch.equal(ph, h[a:b]) and torch.equal(py, y[a:b]), a
