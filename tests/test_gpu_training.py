"""GPU parity: the training operators against their 64-bit formulas.

Tolerances, from the arithmetic alone:
  bf16 outputs   one rounding to 8 bits: 2^-8 of the value (half a unit is 2^-9)
  fp32 sums      K products summed in fp32, each step off by at most 2^-23 of the
                 running sum: K 2^-23 of the sum of the products' magnitudes
  fp32 functions a few operations and fast exp / divide: 1e-5 of the terms' magnitudes
"""
import numpy as np
import pytest
import torch

import _training_ref as ref
import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F64 = torch.float64
BF = torch.bfloat16


def _randn(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def _offsets(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)


def _close(got, want, slack, what):
    """|got - want| <= 2^-8 |want| for bf16 (2^-23 for fp32), plus `slack` elementwise; NaN where NaN is wanted."""
    got, want = got.to(F64), want.to(got.device)
    unit = 2.0 ** -8 if what.startswith("bf16") else 2.0 ** -23
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    ok = ~torch.isnan(want)
    over = ((got - want).abs() - unit * want.abs() - slack)[ok]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: over the bound by {float(over.max()):.3e}"


EDGES = [[0, 1, 127, 128, 129, 0, 255, 256, 300], [1], [0, 0, 5, 0], [257, 511, 513], [16, 15, 17, 64, 63, 65]]


@pytest.mark.parametrize("counts", EDGES)
@pytest.mark.parametrize("n,d,parts", [(64, 64, 1), (192, 320, 2), (384, 256, 1), (128, 576, 2)])
def test_dgrad_edges(counts, n, d, parts):
    S, E = sum(counts), len(counts)
    off = _offsets(counts)
    do = [_randn((S, n), 10 + i) for i in range(parts)]
    w = [_randn((E, n, d), 20 + i, d ** -0.5) for i in range(parts)]
    second = dict(dout2=do[1], w2=w[1]) if parts == 2 else {}
    dx = mk.mk_moe_grouped_dgrad(do[0], off, w[0], **second)
    want = sum(ref.dgrad(a, off, b) for a, b in zip(do, w))
    size = sum(ref.dgrad(a.abs(), off, b.abs()) for a, b in zip(do, w))
    _close(dx, want, parts * n * 2.0 ** -23 * size, "bf16 dx")


def test_dgrad_long_sum_and_repeat():
    """K = 2 x 2048 through several trips of the stage ring; two calls give the same bits."""
    counts, n, d = [300, 40, 700], 2048, 256
    off = _offsets(counts)
    do = [_randn((sum(counts), n), 1 + i) for i in range(2)]
    w = [_randn((3, n, d), 5 + i, d ** -0.5) for i in range(2)]
    ws = torch.empty(256 + 4 * 4, dtype=torch.uint8, device=DEV)
    dx = mk.mk_moe_grouped_dgrad(do[0], off, w[0], do[1], w[1], ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK
    size = sum(ref.dgrad(a.abs(), off, b.abs()) for a, b in zip(do, w))
    _close(dx, sum(ref.dgrad(a, off, b) for a, b in zip(do, w)), 2 * n * 2.0 ** -23 * size, "bf16 dx")
    again = mk.mk_moe_grouped_dgrad(do[0], off, w[0], do[1], w[1], ws=ws)
    assert torch.equal(dx.view(torch.int16), again.view(torch.int16))


def test_dgrad_is_the_gradient_of_the_grouped_gemm():
    """<dx, v> = <dout, forward(v)> for random v (the adjoint of the forward GEMM)."""
    counts, n, d = [100, 0, 37, 260], 192, 256
    off, S = _offsets(counts), sum(counts)
    do, w, v = _randn((S, n), 1), _randn((4, n, d), 2, d ** -0.5), _randn((S, d), 3)
    left = (mk.mk_moe_grouped_dgrad(do, off, w).to(F64) * v.to(F64)).sum()
    right = (do.to(F64) * mk.mk_moe_grouped_gemm(v, off, w).to(F64)).sum()
    # each side rounds its result to bf16: at most 2^-8 of the sum of its products' magnitudes
    scale = (ref.dgrad(do.abs(), off, w.abs()) * v.to(F64).abs()).sum()
    assert abs(float(left - right)) <= 2.0 ** -8 * float(scale)


WCOUNTS = EDGES + [[767, 0, 768, 769, 1], [1537, 2304, 3]]


@pytest.mark.parametrize("counts", WCOUNTS)
@pytest.mark.parametrize("n,d", [(64, 64), (192, 320), (384, 192), (320, 576)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_wgrad_edges(counts, n, d, dtype):
    S, E = sum(counts), len(counts)
    off = _offsets(counts)
    do, x = _randn((S, n), 1), _randn((S, d), 2)
    dw = torch.full((E, n, d), float("nan"), dtype=dtype, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    mk.mk_moe_grouped_wgrad(do, off, x, dw=dw, ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK
    slack = max(counts) * 2.0 ** -23 * ref.wgrad(do.abs(), off, x.abs(), E)
    _close(dw, ref.wgrad(do, off, x, E), slack, "bf16 dw" if dtype == BF else "fp32 dw")
    for e, c in enumerate(counts):
        if c == 0:
            assert not bool(dw[e].any())


def test_wgrad_accumulates_in_fp32():
    counts, n, d = [40, 0, 900, 17], 192, 256
    off, S = _offsets(counts), sum(counts)
    do, x, before = _randn((S, n), 1), _randn((S, d), 2), _randn((4, n, d), 3, dtype=torch.float32)
    dw = before.clone()
    mk.mk_moe_grouped_wgrad(do, off, x, dw=dw, accumulate=True)
    want = before.to(F64) + ref.wgrad(do, off, x, 4)
    slack = 901 * 2.0 ** -23 * (ref.wgrad(do.abs(), off, x.abs(), 4) + before.to(F64).abs())
    _close(dw, want, slack, "fp32 dw")
    assert torch.equal(dw[1], before[1])  # an expert without rows adds nothing
    again = before.clone()
    mk.mk_moe_grouped_wgrad(do, off, x, dw=again, accumulate=True)
    assert torch.equal(dw.view(torch.int32), again.view(torch.int32))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_wgrad_keeps_other_experts_rows_out(bad):
    """NaN and infinities in an expert's rows reach its own gradient only, wherever its block ends in a k-block."""
    counts, n, d = [17, 3, 64, 30, 1, 800], 128, 192
    off, S = _offsets(counts), sum(counts)
    do, x = _randn((S, n), 1), _randn((S, d), 2)
    for broken in (1, 3, 4):
        a, b = ref.spans(off)[broken]
        do2, x2 = do.clone(), x.clone()
        do2[a:b] = bad
        x2[a:b] = bad
        dw = mk.mk_moe_grouped_wgrad(do2, off, x2)
        clean = mk.mk_moe_grouped_wgrad(do, off, x)
        for e in range(len(counts)):
            if e == broken:
                assert not bool(torch.isfinite(dw[e]).any())
            else:
                assert torch.equal(dw[e], clean[e]), (broken, e)


def test_wgrad_long_sum_keeps_fp32_accuracy():
    """20000 rows in one expert: the error stays at fp32 rounding's, not at that of one long truncated sum.

    Sums of 768 rows are 48 MMA steps, each truncating below 2^-23 of the running sum, so at most
    24 * 2^-23 = 2.9e-6 of the result's scale on average; 2e-6 in norm is the bound for 27 such
    chunks of random signs added with rounding (one long sum measures 1e-5 and more)."""
    S, n, d = 20000, 256, 256
    do, x = _randn((S, n), 1), _randn((S, d), 2)
    off = _offsets([S])
    dw = mk.mk_moe_grouped_wgrad(do, off, x).to(F64)
    want = ref.wgrad(do, off, x, 1)
    assert float((dw - want).norm() / want.norm()) <= 2e-6


@pytest.mark.parametrize("counts,n,d", [([20000], 64, 64), ([9000, 0, 3001, 1], 256, 192), ([511, 13000], 64, 256)])
@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, False), (torch.float32, True), (BF, False)])
def test_wgrad_few_long_experts_in_pieces(counts, n, d, dtype, accumulate):
    """Few tiles and long sums: with the workspace of its size function the sum is cut into pieces and
    joined (ragged pieces, experts without any), without it it is not; both within the bounds."""
    S, E = sum(counts), len(counts)
    off = _offsets(counts)
    do, x = _randn((S, n), 1), _randn((S, d), 2)
    size = mk.load_library().mk_moe_grouped_wgrad_workspace_size(S, d, E, n)
    assert size > 256 + 2 * n * d * 4
    before = _randn((E, n, d), 3, dtype=dtype)
    want = ref.wgrad(do, off, x, E) + (before.to(F64) if accumulate else 0)
    slack = max(counts) * 2.0 ** -23 * (ref.wgrad(do.abs(), off, x.abs(), E) + before.to(F64).abs())
    for nbytes in (size, 256):
        ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        dw = before.clone()
        mk.mk_moe_grouped_wgrad(do, off, x, dw=dw, accumulate=accumulate, ws=ws)
        assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK
        _close(dw, want, slack, "bf16 dw" if dtype == BF else "fp32 dw")
        again = before.clone()
        mk.mk_moe_grouped_wgrad(do, off, x, dw=again, accumulate=accumulate, ws=ws)
        assert torch.equal(dw, again)
    bad = off.clone()
    bad[1] = S + 5
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    dw = before.clone()
    mk.mk_moe_grouped_wgrad(do, bad, x, dw=dw, accumulate=accumulate, ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_ERR_BOUNDS and torch.equal(dw, before)


def test_wgrad_without_rows():
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    do, x = torch.empty((0, 64), dtype=BF, device=DEV), torch.empty((0, 128), dtype=BF, device=DEV)
    dw = mk.mk_moe_grouped_wgrad(do, off, x)
    assert dw.shape == (2, 64, 128) and not bool(dw.any())
    kept = torch.full((2, 64, 128), 3.0, device=DEV)
    mk.mk_moe_grouped_wgrad(do, off, x, dw=kept, accumulate=True)
    assert bool((kept == 3.0).all())
    assert mk.mk_moe_grouped_dgrad(do, off, torch.empty((2, 64, 128), dtype=BF, device=DEV)).shape == (0, 128)


@pytest.mark.parametrize("bad", [[0, 25, 40], [1, 10, 30], [0, 31, 30], [0, -1, 30]])
def test_grouped_gradients_reject_bad_offsets(bad):
    """MK_ERR_BOUNDS on the device, the outputs untouched, and the next call on the workspace works."""
    S, n, d, E = 30, 128, 128, 2
    do, x, w = _randn((S, n), 1), _randn((S, d), 2), _randn((E, n, d), 3)
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    off = torch.tensor(bad, dtype=torch.int32, device=DEV)
    dx = torch.full((S, d), 7.0, dtype=BF, device=DEV)
    mk.mk_moe_grouped_dgrad(do, off, w, dx=dx, ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_ERR_BOUNDS
    dw = torch.full((E, n, d), 7.0, device=DEV)
    mk.mk_moe_grouped_wgrad(do, off, x, dw=dw, ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_ERR_BOUNDS
    assert bool((dx == 7.0).all()) and bool((dw == 7.0).all())
    good = _offsets([10, 20])
    mk.mk_moe_grouped_dgrad(do, good, w, dx=dx, ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK
    mk.mk_moe_grouped_wgrad(do, good, x, dw=dw, ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK


def _spiky(shape, seed):
    """Activations over many binades, with zeros, a zero block, subnormals, the largest bf16, NaN and infinities."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(2 * torch.randn(shape, generator=g))
    x = x.to(BF)
    f = x.view(-1)
    f[5::97] = 0
    f[:32] = 0
    if f.numel() >= 256:
        f[32:64] = torch.tensor(2.0 ** -130)
        f[64] = 3.3895313892515355e38
        f[97] = float("nan")
        f[130] = float("inf")
        f[131] = float("-inf")
        f[160:192] = float("nan")
        f[200] = 1e-38
    return x.to(DEV)


def _slots(T, k, seed):
    p = torch.randperm(T * k, generator=torch.Generator().manual_seed(seed))
    return p.to(torch.int32).view(T, k).to(DEV)


@pytest.mark.parametrize("T,d,k", [(1, 64, 1), (3, 64, 8), (129, 192, 3), (50, 1024, 2), (7, 7168, 8)])
def test_ckpt8_round_trip(T, d, k):
    x = _spiky((T, d), T)
    codes, scales = mk.mk_moe_ckpt8_save(x)
    want, q = ref.round8(x)
    assert torch.equal(scales.cpu().to(torch.int64) - 127, q)
    slot = _slots(T, k, 3)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    rows = mk.mk_moe_ckpt8_dispatch(codes, scales, slot, ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK
    got = rows[slot.long().view(-1)].view(T, k, d).cpu().to(F64)
    for j in range(k):
        assert torch.equal(torch.nan_to_num(got[:, j], nan=1.25), torch.nan_to_num(want, nan=1.25))


def test_ckpt8_error_bound():
    """A value in its block's top nine binades is kept within 2^-4 of itself."""
    x = _randn((64, 256), 9)
    codes, scales = mk.mk_moe_ckpt8_save(x)
    slot = torch.arange(64, dtype=torch.int32, device=DEV).view(64, 1)
    back = mk.mk_moe_ckpt8_dispatch(codes, scales, slot).to(F64)
    x = x.to(F64)
    top = x.abs().view(64, 8, 32).amax(2, keepdim=True).expand(64, 8, 32).reshape(64, 256)
    big = x.abs() >= top * 2.0 ** -9
    assert bool(((back - x).abs() <= 2.0 ** -4 * x.abs())[big].all())


def test_ckpt8_dispatch_skips_rows_out_of_range():
    x = _randn((4, 64), 1)
    codes, scales = mk.mk_moe_ckpt8_save(x)
    out = torch.full((8, 64), 5.0, dtype=BF, device=DEV)
    slot = torch.tensor([[0, 1], [2, 8], [-1, 5], [6, 7]], dtype=torch.int32, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    mk.mk_moe_ckpt8_dispatch(codes, scales, slot, x_perm=out, ws=ws)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_ERR_BOUNDS
    assert bool((out[3:5] == 5.0).all())
    assert torch.equal(out[0], out[1]) and not bool((out[5:8] == 5.0).all())


@pytest.mark.parametrize("S,f", [(1, 64), (3, 320), (129, 512), (33, 1024), (17, 1408), (9, 2048), (2, 4160)])
def test_swiglu_checkpoint_forward_and_backward(S, f):
    gate, up = _randn((S, f), 1, 2.0), _randn((S, f), 2)
    dh = _randn((S, f), 3, 0.1)
    w = torch.rand(S, generator=torch.Generator().manual_seed(4)).to(DEV)
    w[0] = 0.0
    h, codes, scales = mk.mk_moe_swiglu_ckpt8(gate, up)
    want = ref.swiglu(gate, up)
    _close(h, want, 1e-5 * want.abs(), "bf16 h")
    g8, qg = ref.round8(gate)
    u8, qu = ref.round8(up)
    assert torch.equal(scales.cpu().to(torch.int64) - 127, torch.stack([qg, qu]))
    g8, u8 = g8.to(DEV), u8.to(DEV)
    for weight in (w, None):
        dgate, dup, hw, drw = mk.mk_moe_swiglu_ckpt8_bwd(dh, codes, scales, weight)
        ww = torch.ones(S, device=DEV) if weight is None else weight
        rg, ru, rh, rw = ref.swiglu_bwd(dh, g8, u8, ww)
        s = torch.special.expit(g8)
        terms = ww.to(F64)[:, None] * (dh.to(F64) * u8).abs() * s * (1 + g8.abs() * (1 - s))
        _close(dgate, rg, 1e-5 * terms, "bf16 dgate")
        _close(dup, ru, 1e-5 * ru.abs(), "bf16 dup")
        _close(hw, rh, 1e-5 * rh.abs(), "bf16 hw")
        _close(drw, rw, 1e-5 * (dh.to(F64) * g8 * s * u8).abs().sum(1), "fp32 drow_weight")


def test_swiglu_extreme_gates():
    """Gates of any size give finite results: silu and its slope go to 0 and 0 on the left, g and 1 on the right."""
    f = 64
    gate = torch.zeros((2, f), dtype=BF, device=DEV)
    gate[0] = torch.linspace(-120, 120, f).to(BF)
    gate[1, :3] = torch.tensor([-3e38, 3e38, -89.0], dtype=BF)
    up = torch.ones((2, f), dtype=BF, device=DEV)
    dh = torch.full((2, f), 1e-3, dtype=BF, device=DEV)
    h, codes, scales = mk.mk_moe_swiglu_ckpt8(gate, up)
    dgate, dup, hw, _ = mk.mk_moe_swiglu_ckpt8_bwd(dh, codes, scales)
    for t in (h, dgate, dup, hw):
        assert bool(torch.isfinite(t).all())
    # silu below -87 is under 2e-36: the fast divide may give 0 there
    _close(h, ref.swiglu(gate, up), 1e-5 * ref.swiglu(gate, up).abs() + 1e-35, "bf16 h")


def test_swiglu_non_finite_values_stay_visible():
    gate, up = _randn((4, 64), 1), _randn((4, 64), 2)
    gate[1, 3] = float("nan")
    up[2, 40] = float("inf")
    dh = _randn((4, 64), 3)
    _, codes, scales = mk.mk_moe_swiglu_ckpt8(gate, up)
    dgate, dup, hw, drw = mk.mk_moe_swiglu_ckpt8_bwd(dh, codes, scales)
    assert bool(torch.isnan(dgate[1, 3])) and bool(torch.isnan(dup[1, 3])) and bool(torch.isnan(hw[2, 40]))
    assert int(torch.isnan(dgate).sum()) == 2 and torch.isnan(drw).tolist() == [False, True, True, False]


NORM_D = [1, 2, 31, 64, 100, 257, 512, 520, 1001, 2048, 4100, 7168, 8192, 8200, 12289, 16384]


@pytest.mark.parametrize("d", NORM_D)
@pytest.mark.parametrize("dtype,T,residual", [(BF, 1, False), (BF, 37, True), (torch.float32, 5, True),
                                              (torch.float32, 641, False)])
def test_layernorm_forward_and_backward(d, dtype, T, residual):
    x = _randn((T, d), d, 2.0, torch.float32).add_(0.5).to(dtype)
    gamma, beta = 1 + _randn((d,), 2, 0.2, torch.float32), _randn((d,), 3, 0.2, torch.float32)
    dy = _randn((T, d), 4, 0.1)
    dres = _randn((T, d), 5, 0.1, dtype) if residual else None
    eps = 1e-5
    y, mean, rstd = mk.mk_moe_layernorm(x, gamma, beta, eps)
    wy, wm, wr = ref.layernorm(x, gamma, beta, eps)
    size = x.to(F64).abs().amax(1, keepdim=True)
    # d values of size |x| summed in fp32, then the same again for the variance; d = 1 has variance 0
    # and rstd = eps^-1/2, which multiplies the rounding of x - mean
    _close(mean, wm, 1e-6 * size[:, 0], "fp32 mean")
    _close(rstd, wr, 1e-5 * wr, "fp32 rstd")
    _close(y, wy, 1e-6 * size * wr[:, None] * gamma.abs() + 1e-5 * (wy.abs() + beta.abs()), "bf16 y")
    dx, dgamma, dbeta = mk.mk_moe_layernorm_bwd(dy, x, gamma, mean, rstd, dres=dres)
    wx, wg, wb = ref.layernorm_bwd(dy, x, gamma, eps, dres)
    xh = ((x.to(F64) - wm[:, None]) * wr[:, None])
    err = 1e-6 * size * wr[:, None] + 1e-5 * xh.abs()  # of the normalised value
    t = dy.to(F64) * gamma.to(F64)
    along = (t * xh).abs().mean(1, keepdim=True)
    slack = wr[:, None] * (1e-5 * (t.abs() + t.abs().mean(1, keepdim=True) + xh.abs() * along)
                           + err * along + xh.abs() * (t.abs() * err).mean(1, keepdim=True))
    if residual:
        slack = slack + 2.0 ** -23 * dres.to(F64).abs()
    _close(dx, wx, slack, "bf16 dx" if dtype == BF else "fp32 dx")
    _close(dgamma, wg, (dy.to(F64).abs() * err).sum(0) + T * 2.0 ** -23 * (dy.to(F64) * xh).abs().sum(0),
           "fp32 dgamma")
    _close(dbeta, wb, T * 2.0 ** -23 * dy.to(F64).abs().sum(0), "fp32 dbeta")


def test_layernorm_many_rows_repeat():
    """More rows than one pass of the backward's blocks; the weights' gradients repeat bit for bit."""
    T, d = 5000, 640
    x, dy = _randn((T, d), 1), _randn((T, d), 2)
    gamma, beta = 1 + _randn((d,), 3, 0.1, torch.float32), _randn((d,), 4, 0.1, torch.float32)
    _, mean, rstd = mk.mk_moe_layernorm(x, gamma, beta)
    a = mk.mk_moe_layernorm_bwd(dy, x, gamma, mean, rstd)
    b = mk.mk_moe_layernorm_bwd(dy, x, gamma, mean, rstd)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    _, wg, wb = ref.layernorm_bwd(dy, x, gamma, 1e-5)
    _close(a[1], wg, T * 2.0 ** -23 * (dy.to(F64).abs() * 6).sum(0), "fp32 dgamma")
    _close(a[2], wb, T * 2.0 ** -23 * dy.to(F64).abs().sum(0), "fp32 dbeta")


@pytest.mark.parametrize("d", [3, 1001, 2048, 12288])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_layernorm_tensors_on_odd_multiples_of_16_bytes(d, dtype):
    """Tensors that start 16 bytes past a multiple of 32, between NaNs: the same arithmetic, so the
    same bits as for tensors on a multiple of 32, and nothing written around the outputs."""
    T = 13

    def inside(src):  # the same values, 16 bytes into a buffer of NaNs
        pad = 16 // src.element_size()
        buf = torch.full((src.numel() + 2 * pad,), float("nan"), dtype=src.dtype, device=DEV)
        view = buf[pad:pad + src.numel()].view(src.shape)
        view.copy_(src)
        assert view.data_ptr() % 32 == 16
        return buf, view

    x, dy, dres = _randn((T, d), 1, 2.0, dtype), _randn((T, d), 2), _randn((T, d), 3, 1.0, dtype)
    gamma, beta = 1 + _randn((d,), 4, 0.1, torch.float32), _randn((d,), 5, 0.1, torch.float32)
    y, mean, rstd = mk.mk_moe_layernorm(x, gamma, beta)
    dx, dgamma, dbeta = mk.mk_moe_layernorm_bwd(dy, x, gamma, mean, rstd, dres=dres)
    (_, x2), (_, dy2), (_, dres2) = inside(x), inside(dy), inside(dres)
    (_, gamma2), (_, beta2) = inside(gamma), inside(beta)
    (ybuf, y2), (dxbuf, dx2) = inside(torch.zeros_like(y)), inside(torch.zeros_like(dx))
    mk.mk_moe_layernorm(x2, gamma2, beta2, y=y2, mean=mean, rstd=rstd)
    _, dgamma2, dbeta2 = mk.mk_moe_layernorm_bwd(dy2, x2, gamma2, mean, rstd, dres=dres2, dx=dx2)
    for got, want in ((y2, y), (dx2, dx), (dgamma2, dgamma), (dbeta2, dbeta)):
        assert torch.equal(got, want)
    for buf, t in ((ybuf, y), (dxbuf, dx)):
        pad = 16 // t.element_size()
        assert bool(torch.isnan(buf[:pad]).all()) and bool(torch.isnan(buf[pad + t.numel():]).all())


def test_layernorm_constant_rows_and_no_rows():
    """A constant row has variance zero: y = beta, finite gradients; no rows give zero weight gradients."""
    d = 96
    x = torch.full((3, d), 2.5, dtype=BF, device=DEV)
    gamma, beta = torch.ones(d, device=DEV), torch.linspace(-1, 1, d).to(DEV)
    y, mean, rstd = mk.mk_moe_layernorm(x, gamma, beta)
    assert torch.equal(y, beta.to(BF).expand(3, d)) and bool((mean == 2.5).all())
    dx, dgamma, _ = mk.mk_moe_layernorm_bwd(_randn((3, d), 1), x, gamma, mean, rstd)
    assert bool(torch.isfinite(dx).all()) and not bool(dgamma.any())
    none = torch.empty((0, d), dtype=BF, device=DEV)
    y, mean, rstd = mk.mk_moe_layernorm(none, gamma, beta)
    dx, dgamma, dbeta = mk.mk_moe_layernorm_bwd(none, none, gamma, mean, rstd)
    assert dx.shape == (0, d) and not bool(dgamma.any()) and not bool(dbeta.any())


def test_calls_run_on_the_given_stream():
    """Work of another stream is waited for by that stream alone: the calls follow it in order."""
    s = torch.cuda.Stream()
    counts, n, d = [33, 0, 100], 128, 192
    off, S = _offsets(counts), sum(counts)
    do, x, w = _randn((S, n), 1), _randn((S, d), 2), _randn((3, n, d), 3)
    gamma, beta = torch.ones(d, device=DEV), torch.zeros(d, device=DEV)
    plain = (mk.mk_moe_grouped_dgrad(do, off, w), mk.mk_moe_grouped_wgrad(do, off, x), mk.mk_moe_layernorm(x, gamma, beta)[0])
    torch.cuda.synchronize()
    late_do, late_x = torch.zeros_like(do), torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late_do.copy_(do)
        late_x.copy_(x)
    got = (mk.mk_moe_grouped_dgrad(late_do, off, w, stream=s), mk.mk_moe_grouped_wgrad(late_do, off, late_x, stream=s),
           mk.mk_moe_layernorm(late_x, gamma, beta, stream=s)[0])
    s.synchronize()
    for p, q in zip(plain, got):
        assert torch.equal(p, q)
